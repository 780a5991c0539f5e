"""How far the gradients of the linear cross entropy are off as a whole (needs a GB300).

Bounds that hold for every entry have to add up magnitudes; over a whole gradient
roundings are independent, and their variances add up.  A rounding to bfloat16 is off by up
to half a step and spread evenly, variance step^2 / 12.  The result's own rounding and those
of dZ's entries (but the labels', which are made good) give the expected square of the
error's norm; other errors (single-precision sums, exponentials: 2^-18 of a term) are far
below it.  The square's own spread is small over so many entries: 1.1 of its root bounds it.
"""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv
import train_ref as ref
from test_gpu_linear_ce import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


def variance(x):
    """step^2 / 12 of a rounding to bfloat16 at x."""
    return torch.where(x == 0, 0.0, torch.ldexp(torch.ones_like(x), torch.frexp(x)[1] - 8).square() / 12)


@pytest.mark.parametrize("N,V,D", [
    (64, 1024, 128), (777, 4003, 1000), (5, 20011, 2048), (300, 9001, 264), (2500, 3001, 512),
    (600, 40000, 64), (1030, 600, 4096),
])
@pytest.mark.parametrize("mean", [False, True])  # one weight for all tokens
def test_relative_error_of_the_gradients(N, V, D, mean):
    h, w, y, g = inputs(N, V, D, seed=N + V + D)
    if mean:
        g.fill_(1.0 / N)
        y[::3] = 17  # a third of the tokens have one label
    ce = sv.LinearCe(h, w, y, g)
    nll, lse = ce.loss()
    dh, dw = ce.grad()
    rh, rw, dz, _ = ref.ce_grad(h, w, y, g)
    rows = torch.nonzero(y >= 0)[:, 0]
    v = variance(dz)
    v[rows, y[rows].long()] = 0.0
    for got, want, a, other in ((dh, rh, v, w), (dw, rw, v.t(), h)):
        expected = float((variance(want) + a @ other.double().square()).sum()) ** 0.5
        floor = 2.0 ** -18 * float(want.norm())
        assert float((got.double() - want).norm()) <= 1.1 * expected + floor
        # And along the gradient itself, where a bias would be.  With R the result's roundings and
        # E those of dZ, <R + E other, want> = <R, want> + <E, want other^T>, whose variance is the
        # sum of each rounding's times the square of what it is multiplied with: six deviations.
        # (A first form took the largest entry of a @ other^2 for the second sum, which is not
        # its variance: the roundings of dZ add up along the gradient.)
        along = float(((got.double() - want) * want).sum())
        var = (variance(want) * want.square()).sum() + (a * (want @ other.double().t()).square()).sum()
        assert abs(along) <= 6 * float(var) ** 0.5 + floor * float(want.norm())
