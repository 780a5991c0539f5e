"""Global norm and clip of entries whose squares overflow only once many are added (needs a GB300).

Single precision holds sums of squares up to 3.4e38: one entry from 1.8e19 on, a thread's
64 from 2.3e18, a warp's 2048 from 4e17, a block's or a tensor's from less.  Tolerances: those of
test_gpu_grad_norm.py.
"""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv
import train_ref as ref
from test_gpu_grad_norm import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


@pytest.mark.parametrize("value", [1e13, 1.3e14, 1.5e14, 2e15, 1e16, 1e17, 3e17, 1e18, 2.4e18, 5e18,
                                   1.5e19, 1.8e19, 1.9e19, 1e20])
@pytest.mark.parametrize("sizes", [[1], [3, 70], [5000, 3], [100003, 17], [3_000_000, 12345]],
                         ids=lambda s: str(max(s)))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_equal_entries(dtype, sizes, value):
    grads = [torch.full((n,), value, device="cuda").to(dtype) for n in sizes]
    before = [t.clone() for t in grads]
    out = [torch.empty_like(t) for t in grads]
    n0 = sv.spec_grad_norm(grads)
    n1 = sv.spec_clip_grad_norm(grads, 1.0, out=out)
    assert bool(torch.isfinite(n0).all())
    check(before, out, n1, 1.0)
    n2 = sv.spec_clip_grad_norm(grads, 1.0)
    check(before, grads, n2, 1.0)
    assert torch.equal(n0, n1) and torch.equal(n1, n2)


@pytest.mark.parametrize("scale", [1e16, 1e18, 4e18])
@pytest.mark.parametrize("n", [4000, 2_000_001])
def test_mixed_entries(n, scale):
    # Threads' sums on both sides of every limit, off a 16-byte line as well.
    g = torch.Generator(device="cuda").manual_seed(n)
    a = torch.randn(n, generator=g, device="cuda") * scale
    b = (torch.randn(n + 1, generator=g, device="cuda") * scale).to(torch.bfloat16)[1:]
    c = torch.randn(n, generator=g, device="cuda")
    group = [a, b, c]
    out = [torch.empty_like(t) for t in group]
    check(group, out, sv.spec_clip_grad_norm(group, 3.0, out=out), 3.0)
    assert abs(float(sv.spec_grad_norm([a])) - ref.norm([a])) <= 2.0 ** -18 * ref.norm([a])
