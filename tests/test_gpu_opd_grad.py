"""Gradient of the mixture distillation loss on the GPU against double precision (needs a GB300).

Tolerance.  Every entry is g/L [q ((1 - a) (u - sum q u) + a) - a [x*]].  In
single precision the exponent of q is off by |log2 q| 2^-24 and its normaliser
by at most 2^-19 (exponentials 2^-22 each, per-thread sums of at most a few
hundred terms, float-float above), t by a few roundings of its operands
(below |log2 q| 2^-22 for these rows) and the same normalisers, sum q u by the
same relative amount of sum q |u| plus its own additions (2^-16 for the
longest per-thread sums).  So an entry is off by at most
  (2^-15 + |ln q| 2^-21) times the magnitude of what is added up in it,
and by half a step of its type.  The gradient jumps where q t passes delta: a
row with an entry within 2e-4 of it (the errors above, over t >= delta) may be on
either side of the jump.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv
from speculative_decoding_verification_58_gb300 import synth
import train_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


def check(t, d, L, g, out, delta=0.01, alpha=0.8):
    half = torch.finfo(out.dtype).eps / 2
    sides = []
    for flip in (0.0, 2e-4):
        want, scale, logq, at_clip = ref.opd_grad(t, d, L, g, delta, alpha, flip)
        tol = scale * (2.0 ** -15 + logq.abs() * 2.0 ** -21) + half * want.abs() + 1e-37
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(out), nan)
        sides.append(((((out.double() - want).abs() <= tol) | nan).all(2), at_clip))
    assert torch.all(sides[0][0] | (sides[1][0] & sides[1][1]))


def device(inp):
    d = sv.to_device(inp)
    g = torch.from_numpy(np.linspace(0.5, 1.5, inp.B).astype(np.float32)).cuda()
    return d["target_logits"], d["draft_logits"], d["lengths"], g


@pytest.mark.parametrize("recipe,B,k,V,dtype,seed", [
    ("gauss", 1, 4, 1024, "f32", 1),
    ("gauss", 2, 3, 1, "bf16", 2),
    ("gauss", 3, 2, 7, "f32", 3),
    ("zipf_mixed_noise", 8, 3, 257, "bf16", 4),       # rows not 16-byte aligned
    ("zipf_mixed_noise", 5, 7, 4099, "f32", 5),
    ("zipf_adaptive", 4, 16, 5000, "bf16", 6),
    ("zipf_adaptive", 4, 8, 32000, "bf16", 7),
    ("zipf_adaptive", 2, 16, 50021, "bf16", 8),
    ("zipf_mixed_noise", 2, 5, 151936, "f32", 9),
    ("zipf_adaptive", 3, 16, 151936, "bf16", 10),
    ("gauss", 1, 31, 70001, "f32", 11),
])
def test_gradient(recipe, B, k, V, dtype, seed):
    t, d, L, g = device(synth.make_inputs(recipe, B, k, V, dtype, seed=400 + seed))
    check(t, d, L, g, sv.spec_opd_grad(t, d, L, g))


@pytest.mark.parametrize("V", [2, 7, 8, 9, 15, 16, 17, 100, 2047, 2049, 16385])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_small_and_ragged_rows(V, dtype):
    t, d, L, g = device(synth.make_inputs("zipf_mixed_noise", 3, 5, V, dtype, seed=500 + V))
    check(t, d, L, g, sv.spec_opd_grad(t, d, L, g))


@pytest.mark.parametrize("B,k,V,dtype", [
    (200, 16, 5003, "bf16"),    # several positions for every cluster, rows that lie differently
    (150, 5, 16385, "f32"),
    (64, 16, 32000, "bf16"),
    (3000, 2, 100, "f32"),      # more requests than are counted out
    (2500, 3, 2049, "bf16"),
])
def test_many_positions(B, k, V, dtype):
    t, d, L, g = device(synth.make_inputs("gauss", B, k, V, dtype, seed=520))
    gen = torch.Generator(device="cuda").manual_seed(B)
    L.copy_(torch.randint(1, k + 1, (B,), generator=gen, device="cuda", dtype=torch.int32))
    L[5], L[B - 1], L[0] = 0, k, 1          # an invalid request among them
    out = sv.spec_opd_grad(t, d, L, g)
    check(t, d, L, g, out)
    assert torch.equal(out.view(torch.int16 if dtype == "bf16" else torch.int32),
                       sv.spec_opd_grad(t, d, L, g).view(
                           torch.int16 if dtype == "bf16" else torch.int32))


@pytest.mark.parametrize("off", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (3, 3, 3), (0, 5, 5), (2, 0, 4)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [777, 1024])
def test_buffers_off_16_byte_lines(off, dtype, V):
    # Contiguous tensors that start anywhere; NaN around the inputs, a mark around the output.
    t, d, L, g = device(synth.make_inputs("zipf_mixed_noise", 4, 3, V, dtype, seed=510))
    out = torch.empty_like(d)
    views, flats = [], []
    for x, o, fill in ((t, off[0], float("nan")), (d, off[1], float("nan")), (out, off[2], 7.0)):
        f = torch.full((x.numel() + 16,), fill, dtype=x.dtype, device="cuda")
        v = f[o:o + x.numel()].view(x.shape)
        if fill != 7.0:
            v.copy_(x)
        views.append(v)
        flats.append(f)
    got = sv.spec_opd_grad(views[0], views[1], L, g, d_draft=views[2])
    check(t, d, L, g, got)
    assert torch.all(flats[2][:off[2]] == 7) and torch.all(flats[2][off[2] + out.numel():] == 7)


@pytest.mark.parametrize("alpha,delta", [(0.0, 0.01), (1.0, 0.01), (0.5, 1e-4), (0.3, 1e9)])
def test_mixture_and_clip(alpha, delta):
    t, d, L, g = device(synth.make_inputs("zipf_mixed_noise", 6, 5, 3000, "f32", seed=421))
    check(t, d, L, g, sv.spec_opd_grad(t, d, L, g, alpha=alpha, delta=delta), delta, alpha)


def test_masked_logits_and_bad_rows():
    t, d, L, g = device(synth.make_inputs("zipf_mixed_noise", 8, 4, 2000, "f32", seed=431))
    L.fill_(4)
    inf = float("inf")
    d[0, 0, 100:400] = -inf                   # the drafter excludes entries
    t[1, 1, 50:300] = -inf                    # the target does: those entries are clipped
    t[2, 2, 7:900], d[2, 2, 500:1200] = -inf, -inf
    d[3, 0, 5] = float("nan")                 # rows without finite mass: NaN positions
    t[3, 1, 9] = inf
    d[3, 2] = -inf
    d[4, 0, :] = torch.finfo(torch.float32).min  # all at the type's lowest value: uniform
    d[5, 1, 1:] = torch.finfo(torch.float32).min  # one entry holds all the mass
    d[6] += 1000.0                            # a shift changes nothing
    out = sv.spec_opd_grad(t, d, L, g)
    assert torch.all(torch.isnan(out[3, :3])) and not torch.any(torch.isnan(out[3, 3]))
    check(t, d, L, g, out)


def test_lengths():
    t, d, L, g = device(synth.make_inputs("gauss", 6, 5, 900, "bf16", seed=441))
    L.copy_(torch.tensor([0, 1, 5, 6, -3, 2], dtype=torch.int32))
    out = sv.spec_opd_grad(t, d, L, g)
    for b in (0, 3, 4):
        assert torch.all(torch.isnan(out[b]))
    assert torch.all(out[1, 1:] == 0) and torch.all(out[5, 2:] == 0)
    check(t, d, L, g, out)


def test_equal_rows_and_ties():
    # p = q: t = 0, u = 1; the hard term pulls towards the lowest argmax.
    t, d, L, g = device(synth.make_inputs("gauss", 2, 3, 500, "f32", seed=451))
    L.fill_(3)
    t[0, :, 17], t[0, :, 300] = 50.0, 50.0
    d.copy_(t[:, :3])
    check(t, d, L, g, sv.spec_opd_grad(t, d, L, g))


def test_every_row_sums_to_zero():
    # The loss does not change when a row is shifted: the gradient sums to 0
    # up to half a step of each entry.
    t, d, L, g = device(synth.make_inputs("zipf_adaptive", 4, 6, 32000, "f32", seed=461))
    out = sv.spec_opd_grad(t, d, L, g).double()
    assert torch.all(out.sum(2).abs() <= 2.0 ** -15 * (out.abs().sum(2) + 1e-30) * 4)


def test_against_differences_of_the_loss():
    # The library's own loss in single precision has an error of about 3e-5
    # absolute (its own test); a step of 0.05 along a random direction moves it by
    # about 0.05 |grad . d|, and the central difference is off by O(0.05^2).
    t, d, L, g = device(synth.make_inputs("gauss", 3, 3, 64, "f32", seed=471))
    L.copy_(torch.tensor([3, 2, 1], dtype=torch.int32))
    out = sv.spec_opd_grad(t, d, L, g, delta=1e9)
    gen = torch.Generator(device="cuda").manual_seed(3)
    v = torch.randn(d.shape, generator=gen, device="cuda")
    f = [float((ref.opd_loss(t, d.double() + s * 1e-5 * v.double(), L, 1e9, 0.8) *
                g.double()).sum()) for s in (1, -1)]
    got = float((out.double() * v.double()).sum())
    # Central difference in double precision: O(1e-10) and 1e-16 / 1e-5 of rounding.
    tol = 2.0 ** -14 * float((out.double() * v.double()).abs().sum()) + 1e-8
    assert abs(got - (f[0] - f[1]) / 2e-5) <= tol
    # And the library's own loss moves with it.
    h = 0.02
    st = [sv.spec_opd_stats(t, (d + s * h * v).contiguous(), L, delta=1e9).loss.double()
          for s in (1, -1)]
    own = float(((st[0] - st[1]) / (2 * h) * g.double()).sum())
    assert abs(got - own) <= 4 * 3e-5 * float(g.sum()) / h + 0.05 * abs(got) + 0.05


def test_stream_and_graph():
    t, d, L, g = device(synth.make_inputs("zipf_adaptive", 4, 4, 8000, "bf16", seed=481))
    first = sv.spec_opd_grad(t, d, L, g).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    second = sv.spec_opd_grad(t, d, L, g, stream=s)
    s.synchronize()
    assert torch.equal(first, second)
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_opd_grad(t, d, L, g, d_draft=out)
    t2, d2, L2, g2 = device(synth.make_inputs("zipf_adaptive", 4, 4, 8000, "bf16", seed=482))
    for x, y in ((t, t2), (d, d2), (L, L2), (g, g2)):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    check(t2, d2, L2, g2, out)


def test_refusals():
    t, d, L, g = device(synth.make_inputs("gauss", 2, 3, 64, "f32", seed=491))
    for kw in (dict(delta=0.0), dict(delta=float("inf")), dict(alpha=-0.1), dict(alpha=1.5),
               dict(d_draft=d)):
        with pytest.raises(sv.SpecVerifyError) as e:
            sv.spec_opd_grad(t, d, L, g, **kw)
        assert e.value.code == sv.SPEC_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        sv.spec_opd_grad(t, d[:, :2], L, g)
    with pytest.raises(TypeError):
        sv.spec_opd_grad(t, d.to(torch.bfloat16), L, g)
    with pytest.raises(TypeError):
        sv.spec_opd_grad(t, d, L, g.double())
    with pytest.raises(sv.SpecVerifyError) as e:  # host logits are refused, as by the statistics
        sv.spec_opd_grad(t.cpu().pin_memory(), d.cpu().pin_memory(), L, g)
    assert e.value.code == sv.SPEC_ERR_INVALID_ARG
