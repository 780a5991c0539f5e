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
from test_gpu_linear_ce import check_grad, check_loss, inputs

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


@pytest.mark.parametrize("n,D", [(1, 1024), (1, 4096), (2, 2048), (3, 1000), (4, 1024)])
def test_losses_of_a_few_tokens_have_no_bias(n, D):
    V = 3000
    h, w, y = leaning(96, V, D, seed=D + n)
    nll, lse = (torch.cat(x) for x in zip(*[sv.spec_linear_ce(h[i:i + n].contiguous(), w,
                                                              y[i:i + n].contiguous())
                                            for i in range(0, 96, n)]))
    rn, rl = ref.ce(h, w, y)
    # Absolute, for lse as for the loss: half a step of the logit (2^-24 of 16) for each of the
    # two logits that count, and the approximate exponentials and logarithms (2^-22).
    bound = 2 * 2.0 ** -24 * float((h.double() @ w.double().t()).max()) + 2.0 ** -22
    assert abs(float((lse.double() - rl).mean())) <= bound
    # The losses are small (nearly all mass at the label), so that what is left of them is
    # relative: the errors of both logits, the other entries' exponentials and sums.
    rel = (nll.double() - rn) / rn
    assert abs(float(rel.mean())) <= bound + 2.0 ** -21


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


@pytest.mark.parametrize("N", range(1, 18))
def test_few_tokens(N):
    for V, D in ((1, 8), (300, 72), (5001, 1032), (257, 2056)):
        h, w, y, g = inputs(N, V, D, seed=100 * N + D)
        y[0] = V - 1
        if N > 2:
            y[1], y[2] = 0, -1
        ce = sv.LinearCe(h, w, y, g)
        nll, lse = ce.loss()
        check_loss(h, w, y, nll, lse)
        check_grad(h, w, y, g, *ce.grad())
        one = [sv.spec_linear_ce(h[i:i + 1].contiguous(), w, y[i:i + 1].contiguous())
               for i in range(N)]
        check_loss(h, w, y, torch.cat([a for a, _ in one]), torch.cat([b for _, b in one]))
    if N > 2:  # a bad token spoils its own results only
        h[1, 3] = float("nan")
        nll, lse = sv.spec_linear_ce(h, w, y)
        assert torch.isnan(lse).nonzero().tolist() == [[1]]
        keep = torch.arange(N, device="cuda") != 1
        check_loss(h[keep], w, y[keep], nll[keep], lse[keep])


def test_probabilities_of_a_wide_head_sum_to_one():
    # With a column of ones in the weight, that column of dH is g sum_v (p_v - [v = y]) = 0: what
    # is there is what z, formed again, is off against lse.  All logits are about 16, sums of
    # one sign over D = 8192.
    N, V, D = 256, 4096, 8192
    gen = torch.Generator(device="cuda").manual_seed(5)
    w = (0.5 + torch.rand((V, D), generator=gen, device="cuda")).to(torch.bfloat16)
    w[:, 0] = 1.0
    h = (16.0 / D * 2 * torch.rand((N, D), generator=gen, device="cuda")).to(torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    nll, lse = sv.spec_linear_ce(h, w, y)
    dh, _ = sv.spec_linear_ce_grad(h, w, y, nll, lse, torch.ones(N, device="cuda"), need_weight=False)
    # The means of N V roundings of dZ's entries (2^-8 of 1 / V at most, of random sign), six
    # deviations; two logits' sums of eight chunks (2^-21 of themselves each, as above).
    noise = 6 * 2.0 ** -8 / 3.0 ** 0.5 / (N * V) ** 0.5
    top = float((h.double() @ w.double().t()).max())
    assert abs(float(dh[:, 0].double().mean())) <= noise + 2.0 ** -21 * top / 4 + 2.0 ** -20


@pytest.mark.parametrize("N,D", [(262144, 1024), (100000, 136)])
def test_weight_gradients_of_very_many_tokens(N, D):
    # W = 0: every entry of dZ but the labels' is 1 / V exactly, and a row of dW without labels
    # the mean of the hidden states, all positive.  A cut takes less than a step (2^-23) of the
    # running sum, which over a chunk of 4096 steps is half its end on average: 2^-12 of it.
    V = 64
    gen = torch.Generator(device="cuda").manual_seed(N)
    scale = 0.5 + torch.rand((1, D), generator=gen, device="cuda")
    h = (torch.rand((N, D), generator=gen, device="cuda") * scale).to(torch.bfloat16)
    w = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    y = (torch.arange(N, device="cuda") % 3).to(torch.int32)
    ce = sv.LinearCe(h, w, y, torch.ones(N, device="cuda"), need_hidden=False)
    ce.loss()
    _, dw = ce.grad()
    want = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    for r in range(0, N, 8192):
        part = h[r:r + 8192].double()
        want += part.sum(0) / V
        for k in range(3):
            want[k] -= part[y[r:r + 8192] == k].sum(0)
    err = (dw.double() - want).abs()
    assert torch.all(err <= (2.0 ** -8 + 2.0 ** -12 + 2.0 ** -18) * want.abs())
    row, x = want[5], dw[5].double()
    step = torch.ldexp(torch.ones_like(row), torch.frexp(row)[1] - 9)
    noise = 6 * float((step * row).square().sum().sqrt() / row.square().sum()) / 3.0 ** 0.5
    assert abs(float(((x - row) * row).sum() / row.square().sum())) <= 2.0 ** -12 + noise
