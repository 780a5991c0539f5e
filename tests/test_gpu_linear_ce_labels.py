"""Gradients of the linear cross entropy where many tokens share a label (needs a GB300).

The label's entry of dZ is rounded to bfloat16 for the products, and what the rounding
takes is added back in single precision, so it may not show: an entry of dW or dH is off by
half a step of its own (computed from its binade), by the roundings of the *other*
entries of dZ (2^-8 of each at most), by their exponents' error e and by the sums in single
precision (2^-23 of the sum of magnitudes for each term and step).  e: as in
test_gpu_linear_ce.py.
"""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv
import train_ref as ref
from test_gpu_linear_ce import z_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


def half_step(x):
    """Half the distance of bfloat16 numbers around |x|."""
    return torch.ldexp(torch.ones_like(x), torch.frexp(x)[1] - 9)


def check_tight(h, w, y, g, dh, dw):
    rh, rw, dz, mass = ref.ce_grad(h, w, y, g)
    rows = torch.nonzero((y >= 0) & (y < w.shape[0]))[:, 0]
    rest, label = dz.abs(), torch.zeros_like(dz)
    rest[rows, y[rows].long()] = 0.0
    label[rows, y[rows].long()] = dz[rows, y[rows].long()].abs()
    e = z_error(h, w) + 2.0 ** -18
    for got, want, a, b, m, other in ((dh, rh, rest, label, mass, w.double().abs()),
                                      (dw, rw, rest.t(), label.t(), mass.t(), h.double().abs())):
        K = a.shape[1]
        # exp(-nll) - 1 and its residual: a few roundings of single precision.
        err = (2.0 ** -8 + (K + 8) * 2.0 ** -23) * (a @ other) + \
            ((K + 8) * 2.0 ** -23 + 2.0 ** -20) * (b @ other) + e * (m @ other)
        tol = half_step(want.abs() + err) + err
        assert torch.all((got.double() - want).abs() <= tol + 1e-38)
    return rw, err


def badly_predicted(N, V, D, labels, seed, g):
    """Hidden states with a common part, far from their labels' rows; one weight for all tokens.

    Small products: 2^-23 D max |h| |w| stays below 2^-14."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn((V, D), generator=gen, device="cuda") * (1.0 / D ** 0.5)).to(torch.bfloat16)
    y = labels(torch.arange(N, device="cuda")).to(torch.int32)
    h = 0.5 * torch.randn((N, D), generator=gen, device="cuda") + 0.5 - 3.0 * w[y.long()].float()
    return h.to(torch.bfloat16), w, y, torch.full((N,), g, device="cuda")


# 1 + 2^-8 + 2^-12 lies just above the middle of two bfloat16 numbers: off by 2^-8 rounded.
G = (1.0 + 2.0 ** -8 + 2.0 ** -12) / 64


@pytest.mark.parametrize("N,V,D,labels", [
    (60, 2000, 64, lambda i: torch.full_like(i, 7)),                  # all tokens have one label
    (300, 2000, 136, lambda i: torch.where(i % 5 == 0, 1999, i)),     # every fifth has it
    (700, 4000, 64, lambda i: 640 + i % 32),                          # every row of a block of 32
    (700, 4000, 72, lambda i: (i % 7) * 500 + (i % 3)),               # labels of 33 tokens each
    (40, 3000, 264, lambda i: i // 5),                                # one more than are kept
    (2100, 3000, 64, lambda i: torch.where(i % 2 == 0, 31, i)),       # over more words than a warp has
    (1500, 151936, 64, lambda i: torch.where(i % 3 == 0, 151935, i)), # in the last of several pieces
], ids=["all", "fifth", "block", "few_labels", "five_each", "words", "pieces"])
def test_frequent_labels_under_a_mean_loss(N, V, D, labels):
    h, w, y, g = badly_predicted(N, V, D, labels, seed=N + D, g=G)
    ce = sv.LinearCe(h, w, y, g)
    ce.loss()
    dh, dw = ce.grad()
    rw, err = check_tight(h, w, y, g, dh, dw)
    # The frequent label's row keeps its length: single entries' roundings average out.
    top = int(torch.bincount(y.long(), minlength=V).argmax())
    want, err = rw[top], err[top]
    along = float(((dw[top].double() - want) * want).sum() / want.square().sum())
    # Half steps of the entries, spread evenly: 6 standard deviations; and what is left (above).
    sd = float((half_step(want) * want).square().sum().sqrt() / want.square().sum()) / 3.0 ** 0.5
    assert abs(along) <= 6 * sd + float((err * want.abs()).sum() / want.square().sum())


def test_same_bits_whatever_else_is_wanted():
    h, w, y, g = badly_predicted(400, 1000, 136, lambda i: torch.where(i % 3 == 0, 5, i), 3, G)
    nll, lse = sv.spec_linear_ce(h, w, y)
    _, a = sv.spec_linear_ce_grad(h, w, y, nll, lse, g)
    _, b = sv.spec_linear_ce_grad(h, w, y, nll, lse, g, need_hidden=False)
    assert torch.equal(a, b)
