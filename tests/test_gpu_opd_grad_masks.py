"""The mixture loss's gradient where the target masks entries with finite values (needs a GB300).

A mask that is a finite number, down to the type's lowest, makes log q - log p of a
masked entry a number of that size where the drafter does not mask it.  The clip
holds such an entry constant, so it must leave nothing in the gradient of the others.
Tolerances: those of test_gpu_opd_grad.py; the magnitude of what is added up does not hold
clipped entries, so nothing here widens them.
"""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv
from speculative_decoding_verification_58_gb300 import synth
from test_gpu_opd_grad import check, device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


def off_the_line(x, by):
    """The same contiguous values, `by` entries off a 16-byte line."""
    f = torch.empty(x.numel() + 16, dtype=x.dtype, device=x.device)
    v = f[by:by + x.numel()].view(x.shape)
    v.copy_(x)
    return v


MASKS = [-1e4, -65504.0, -1e5, -1e9, -1e30, None]  # None: the type's lowest


@pytest.mark.parametrize("V", [2000, 4099])
@pytest.mark.parametrize("aligned", [True, False])  # rows in shared memory / read in every pass
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_target_masks(dtype, mask, aligned, V):
    t, d, L, g = device(synth.make_inputs("zipf_mixed_noise", 6, 4, V, dtype, seed=601))
    L.fill_(4)
    low = torch.finfo(t.dtype).min if mask is None else mask
    gen = torch.Generator().manual_seed(8)
    tenth = (torch.rand(t.shape, generator=gen) < 0.1).cuda()
    t[0][tenth[0]] = low                      # the target alone
    t[1][tenth[1]] = low                      # both, partly the same entries
    d[1][tenth[2, :4]] = low
    t[2, :, V // 2:], d[2, :, V // 2:] = low, low  # the same half
    t[3, :, :V // 3] = low                    # a whole stretch, which starts the row
    t[4, 1, :] = low                          # a row at one value is uniform
    t[5, 2, :], t[5, 2, 3] = low, 1.0         # one entry holds all the mass
    if not aligned:
        t, d = off_the_line(t, 1), off_the_line(d, 1)
    check(t, d, L, g, sv.spec_opd_grad(t, d, L, g))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mask", [-1e9, None])
def test_full_vocabulary(dtype, mask):
    # bf16 rows lie in shared memory over a cluster, float rows are read in every pass.
    t, d, L, g = device(synth.make_inputs("zipf_adaptive", 2, 3, 151936, dtype, seed=602))
    low = torch.finfo(t.dtype).min if mask is None else mask
    t[0, :, 1::7] = low
    t[1, :, 140000:], d[1, :, 140000:] = low, low
    check(t, d, L, g, sv.spec_opd_grad(t, d, L, g))


def test_moderate_differences():
    # log q - log p of single entries around the size up to which the sum over all entries
    # is used, and far above it.
    t, d, L, g = device(synth.make_inputs("zipf_mixed_noise", 1, 8, 3000, "f32", seed=603))
    L.fill_(8)
    for i, x in enumerate((10.0, 25.0, 31.0, 33.0, 40.0, 60.0, 200.0, 2000.0)):
        top = d[0, i].topk(40).indices
        t[0, i, top] = d[0, i, top] - x
    check(t, d, L, g, sv.spec_opd_grad(t, d, L, g))
