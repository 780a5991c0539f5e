"""Long sums of the linear cross entropy keep single precision (needs a GB300).

The tensor cores cut a sum off towards zero at every step, which rounding to nearest does
not: over a long sum of one sign that is a bias (of 64 steps, measured: 3e-7 of the sum;
a correctly rounded sum has none).  These tests look at means over many tokens, in
which roundings to nearest average out and a bias stays.
"""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv
import train_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


def leaning(N, V, D, seed):
    """Hidden states that lean on their label's row: its logit is about 16, a sum of one sign."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn((V, D), generator=g, device="cuda") / D ** 0.5).to(torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    h = (16.0 * w[y.long()].float() +
         0.5 * torch.randn((N, D), generator=g, device="cuda")).to(torch.bfloat16)
    return h, w, y


@pytest.mark.parametrize("N,D", [(300, 1024), (64, 4096)])
def test_the_labels_logit_is_rounded_to_nearest(N, D):
    h, w, y = leaning(N, 2000, D, seed=N)
    nll, _ = sv.spec_linear_ce(h, w, y)
    rn, _ = ref.ce(h, w, y)
    z = h.double() @ w.double().t()
    others = z.scatter(1, y.long()[:, None], float("-inf")).amax(1).abs().max()
    # The other entries' logits (of up to 64 steps in one chunk: 2^-21 of themselves), the
    # label's (2^-24 of itself) and the approximate functions.
    bound = 2.0 ** -21 * float(others) + 2.0 ** -24 * float(z.max()) + 2.0 ** -21
    assert abs(float(((nll.double() - rn) / rn).mean())) <= bound
