"""Linear cross entropy and its gradients on the GPU against double precision (needs a GB300).

Tolerances.  A bfloat16 product is exact in single precision; a sum of D of
them in single precision, in any order and rounded to nearest or towards zero,
is off by at most D 2^-23 times the sum of their magnitudes, so a logit by
  e_z = D 2^-23 max_v sum_d |h_d w_vd|.
The exponentials (2^-22 relative), the sums of exponentials (2^-19 covers a
tile's 256 terms added in sequence and the float-float sum above) and the final
log and sums (a few 2^-24 of |lse|) add to it.  dZ is rounded to bfloat16
(2^-8 of its value), has e_z + 2^-19 in the exponent, and the products' sums
are as above; the result is rounded to bfloat16 once more.
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


def inputs(N, V, D, seed=0, lean=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn((V, D), generator=g, device="cuda") * (2.0 / D ** 0.5)).to(torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=g, device="cuda")
    h = torch.randn((N, D), generator=g, device="cuda")
    h = (h + lean * (torch.rand((N, 1), generator=g, device="cuda") < 0.5) * w[y].float())
    skip = torch.rand(N, generator=g, device="cuda") < 0.2
    labels = torch.where(skip, torch.full_like(y, -100), y).to(torch.int32)
    gn = torch.rand(N, generator=g, device="cuda") / N
    return h.to(torch.bfloat16), w, labels, gn


def z_error(h, w):
    # |h| . |w| is largest for one (token, entry) pair; a bound for all.
    top = float((h.double().abs() @ w.double().abs().t()).max())
    return h.shape[1] * 2.0 ** -23 * top


def check_loss(h, w, y, nll, lse):
    rn, rl = ref.ce(h, w, y)
    ez = z_error(h, w)
    tol = ez + 2.0 ** -18 + 2.0 ** -22 * rl.abs()
    assert torch.all((lse.double() - rl).abs() <= tol)
    bad = torch.isnan(rn)
    assert torch.equal(torch.isnan(nll), bad)
    assert torch.all(((nll.double() - rn).abs() <= tol + ez)[~bad])


def check_grad(h, w, y, g, dh, dw):
    rh, rw, dz, mass = ref.ce_grad(h, w, y, g)
    half = 2.0 ** -8
    e = z_error(h, w) + 2.0 ** -18
    for got, want, a, b in ((dh, rh, w, None), (dw, rw, None, h)):
        if got is None:
            continue
        absdz = dz.abs() if b is None else dz.abs().t()
        m = mass if b is None else mass.t()
        other = (w if b is None else h).double().abs()
        K = absdz.shape[1]
        tol = (half + (K + 8) * 2.0 ** -23) * (absdz @ other) + e * (m @ other) + half * want.abs()
        assert torch.all((got.double() - want).abs() <= tol * 1.0001 + 1e-38)


SHAPES = [
    (1, 1, 8), (1, 2, 8), (1, 1000, 64), (2, 63, 72), (3, 257, 128), (17, 1024, 128),
    (64, 4099, 200), (127, 300, 64), (128, 256, 64), (129, 513, 1000), (256, 512, 256),
    (300, 9001, 264), (511, 2047, 512), (1030, 8193, 136), (5, 20011, 4096),
]


@pytest.mark.parametrize("N,V,D", SHAPES)
def test_loss_and_gradients(N, V, D):
    h, w, y, g = inputs(N, V, D, seed=N + V + D)
    y[0] = V - 1  # the last entry of a ragged vocabulary
    ce = sv.LinearCe(h, w, y, g)
    nll, lse = ce.loss()
    dh, dw = ce.grad()
    check_loss(h, w, y, nll, lse)
    check_grad(h, w, y, g, dh, dw)
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_OK


@pytest.mark.parametrize("N,V,D", [(5, 151936, 64), (200, 151936, 128)])
def test_full_vocabulary(N, V, D):
    h, w, y, g = inputs(N, V, D, seed=7)
    ce = sv.LinearCe(h, w, y, g)
    nll, lse = ce.loss()
    dh, dw = ce.grad()
    check_loss(h, w, y, nll, lse)
    check_grad(h, w, y, g, dh, dw)


@pytest.mark.parametrize("N,V,D", [
    (600, 151936, 64),    # two pieces of the vocabulary, slices past the end of the second
    (1030, 100003, 72),
    (2300, 40001, 200),   # dH from one slice, two pieces
])
def test_several_pieces(N, V, D):
    h, w, y, g = inputs(N, V, D, seed=8)
    y[:3] = torch.tensor([0, V - 1, V // 2], dtype=torch.int32)
    ce = sv.LinearCe(h, w, y, g)
    nll, lse = ce.loss()
    dh, dw = ce.grad()
    check_loss(h, w, y, nll, lse)
    check_grad(h, w, y, g, dh, dw)


@pytest.mark.parametrize("N,V,D", [(3001, 300, 64), (9000, 100, 72), (1500, 1, 64), (4097, 257, 8)])
def test_many_tokens_of_few_entries(N, V, D):
    # Every entry is the label of more tokens than are kept for one; the map of labels
    # is longer than a warp.
    h, w, y, g = inputs(N, V, D, seed=12)
    y[N // 2:] = 0
    ce = sv.LinearCe(h, w, y, g)
    nll, lse = ce.loss()
    dh, dw = ce.grad()
    check_loss(h, w, y, nll, lse)
    check_grad(h, w, y, g, dh, dw)


def test_inputs_inside_larger_buffers():
    # Rows of larger tensors as inputs; what surrounds them is NaN.
    N, V, D = 77, 900, 136
    h, w, y, g = inputs(N, V, D, seed=14)
    fh = torch.full((N + 40, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fw = torch.full((V + 300, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fy = torch.full((N + 9,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    fg = torch.full((N + 9,), float("nan"), device="cuda")
    fh[5:5 + N], fw[7:7 + V], fy[3:3 + N], fg[1:1 + N] = h, w, y, g
    ce = sv.LinearCe(fh[5:5 + N], fw[7:7 + V], fy[3:3 + N], fg[1:1 + N])
    nll, lse = ce.loss()
    dh, dw = ce.grad()
    check_loss(h, w, y, nll, lse)
    check_grad(h, w, y, g, dh, dw)
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_OK


def test_one_gradient_alone_is_the_same():
    h, w, y, g = inputs(150, 9000, 128, seed=3)
    ce = sv.LinearCe(h, w, y, g)
    nll, lse = ce.loss()
    dh, dw = ce.grad()
    dh1, none = sv.spec_linear_ce_grad(h, w, y, nll, lse, g, need_weight=False)
    assert none is None and torch.equal(dh, dh1)
    none, dw1 = sv.spec_linear_ce_grad(h, w, y, nll, lse, g, need_hidden=False)
    assert none is None and torch.equal(dw, dw1)


def test_no_token_has_a_label():
    h, w, y, g = inputs(70, 500, 64)
    y.fill_(-1)
    g.fill_(float("nan"))  # not read
    ce = sv.LinearCe(h, w, y, g)
    nll, lse = ce.loss()
    dh, dw = ce.grad()
    assert torch.all(nll == 0) and torch.all(dh == 0) and torch.all(dw == 0)
    assert torch.allclose(lse.double(), ref.ce(h, w, y)[1], atol=1e-4)


def test_label_outside_the_vocabulary():
    h, w, y, g = inputs(40, 300, 64, seed=5)
    y[:4] = 3
    y[1], y[2] = 300, 2 ** 31 - 1
    ce = sv.LinearCe(h, w, y, g)
    nll, lse = ce.loss()
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_ERR_BAD_INPUT
    check_loss(h, w, y, nll, lse)
    dh, dw = ce.grad()
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_ERR_BAD_INPUT
    assert torch.all(dh[1] == 0) and torch.all(dh[2] == 0)
    check_grad(h, w, y, g, dh, dw)


def test_peaked_and_extreme_logits():
    # Logits up to about +-2000: one probability is 1, the others vanish.
    h, w, y, g = inputs(33, 1000, 64, seed=9, lean=0.0)
    h[:8] *= 300
    ce = sv.LinearCe(h, w, y, g)
    nll, lse = ce.loss()
    dh, dw = ce.grad()
    check_loss(h, w, y, nll, lse)
    check_grad(h, w, y, g, dh, dw)


def test_well_predicted_tokens():
    # Every label's probability is within 1e-2 .. 1e-7 of 1: the loss and the
    # gradient keep their relative precision up to that of the logits themselves.
    h, w, y, g = inputs(64, 500, 64, seed=10)
    y = torch.arange(64, device="cuda", dtype=torch.int32)
    lean = torch.linspace(3.5, 6.5, 64, device="cuda")[:, None]
    h = (0.1 * h.float() + lean * w[:64].float()).to(torch.bfloat16)
    ce = sv.LinearCe(h, w, y, g)
    nll, lse = ce.loss()
    dh, dw = ce.grad()
    check_loss(h, w, y, nll, lse)
    check_grad(h, w, y, g, dh, dw)
    rn, _ = ref.ce(h, w, y)
    # log(1 + sum exp(z_v - z_y)): the logits' errors and those of the exponentials
    # and sums (2^-18, above) are relative in it.
    assert torch.all((nll.double() - rn).abs() <= (2.1 * z_error(h, w) + 2.0 ** -18) * rn)
    rh, rw, dz, _ = ref.ce_grad(h, w, y, g)
    tol = (2.0 ** -7 + 4 * z_error(h, w) + 2.0 ** -16) * (dz.abs() @ w.double().abs())
    assert torch.all((dh.double() - rh).abs() <= tol)


def test_not_finite_hidden_state_spoils_its_own_row_only():
    h, w, y, g = inputs(20, 700, 64, seed=11)
    h[3, 5] = float("nan")
    h[4, 0] = float("inf")
    nll, lse = sv.spec_linear_ce(h, w, y)
    bad = torch.isnan(lse)
    assert bad[3] and bad[4] and int(bad.sum()) == 2
    keep = ~bad
    rn, rl = ref.ce(h[keep], w, y[keep])
    assert torch.allclose(lse[keep].double(), rl, atol=1e-4)
    assert torch.allclose(nll[keep].double(), rn, atol=1e-4)


def test_rows_past_the_buffers_are_untouched():
    # Outputs inside larger buffers: nothing before or after them is written.
    N, V, D = 131, 777, 72
    h, w, y, g = inputs(N, V, D, seed=13)
    fh = torch.full((N + 300, D), 7.0, dtype=torch.bfloat16, device="cuda")
    fw = torch.full((V + 600, D), 7.0, dtype=torch.bfloat16, device="cuda")
    fl = torch.full((2, N + 64), 7.0, device="cuda")
    ce = sv.LinearCe(h, w, y, g, nll=fl[0, 8:8 + N], lse=fl[1, 8:8 + N], d_hidden=fh[100:100 + N],
                     d_weight=fw[200:200 + V])
    nll, lse = ce.loss()
    dh, dw = ce.grad()
    check_loss(h, w, y, nll, lse)
    check_grad(h, w, y, g, dh, dw)
    for f, a, n in ((fh, 100, N), (fw, 200, V)):
        assert torch.all(f[:a] == 7) and torch.all(f[a + n:] == 7)
    assert torch.all(fl[:, :8] == 7) and torch.all(fl[:, 8 + N:] == 7)


def test_same_bits_again_and_on_another_stream():
    h, w, y, g = inputs(260, 5003, 136, seed=15)
    first = [t.clone() for t in sv.LinearCe(h, w, y, g).loss()]
    a = sv.LinearCe(h, w, y, g)
    a.loss()
    ga = [t.clone() for t in a.grad()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = sv.LinearCe(h, w, y, g, stream=s)
    c = sv.LinearCe(h, w, y, g)  # beside it on the current stream, own workspace
    for _ in range(3):
        lb = b.loss()
        c.loss()
        gb = b.grad()
        gc = c.grad()
    torch.cuda.synchronize()
    for x, z in zip(first + ga + ga, list(lb) + list(gb) + list(gc)):
        assert torch.equal(x, z)


def test_graph_replay_reads_new_contents():
    h, w, y, g = inputs(100, 3000, 64, seed=17)
    ce = sv.LinearCe(h, w, y, g)
    ce.loss(), ce.grad()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        cap = sv.LinearCe(h, w, y, g, nll=ce.nll, lse=ce.lse, d_hidden=ce.d_hidden,
                          d_weight=ce.d_weight, workspace=ce.workspace)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            cap.loss()
            cap.grad()
    h2, w2, y2, g2 = inputs(100, 3000, 64, seed=18)
    for dst, src in ((h, h2), (w, w2), (y, y2), (g, g2)):
        dst.copy_(src)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    check_loss(h2, w2, y2, ce.nll, ce.lse)
    check_grad(h2, w2, y2, g2, ce.d_hidden, ce.d_weight)


def test_gradients_against_differences():
    # Directional difference of the double-precision loss at the bfloat16
    # inputs: (f(x + e d) - f(x - e d)) / 2e is off by O(e^2); e = 1e-4 keeps
    # that and the cancellation below 1e-6 of the sum of magnitudes.
    h, w, y, g = inputs(9, 50, 16, seed=19)
    ce = sv.LinearCe(h, w, y, g)
    ce.loss()
    dh, dw = ce.grad()
    gd = g.double()
    gen = torch.Generator(device="cuda").manual_seed(1)
    for x, grad, at in ((h, dh, 0), (w, dw, 1)):
        d = torch.randn(x.shape, generator=gen, device="cuda", dtype=torch.float64)
        f = []
        for sgn in (1, -1):
            xs = [h.double(), w.double()]
            xs[at] = xs[at] + sgn * 1e-4 * d
            f.append(float((ref.ce(xs[0], xs[1], y)[0] * gd).sum()))
        diff = (f[0] - f[1]) / 2e-4
        got = float((grad.double() * d).sum())
        # Two roundings to bfloat16 (2^-8 each) of every term.
        tol = 2.0 ** -7 * float((grad.double() * d).abs().sum()) + \
            2.0 ** -8 * float(gd.sum()) * float(d.abs().max()) * float(x.double().abs().max()) * 16
        assert abs(got - diff) <= tol


def test_refusals():
    h, w, y, g = inputs(8, 40, 16)
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.spec_linear_ce(h.float(), w.float(), y)
    assert e.value.code == sv.SPEC_ERR_UNSUPPORTED
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.spec_linear_ce(h[:, :12].contiguous(), w[:, :12].contiguous(), y)
    assert e.value.code == sv.SPEC_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        sv.spec_linear_ce(h[:, :8], w[:, :8], y)          # not contiguous
    with pytest.raises(TypeError):
        sv.spec_linear_ce(h, w, y.long())
    with pytest.raises(TypeError):
        sv.spec_linear_ce(h, w.float(), y)
    with pytest.raises(ValueError):
        sv.spec_linear_ce(h, w, y[:4])
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.spec_linear_ce(h, w, y, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == sv.SPEC_ERR_WORKSPACE
    nll, lse = sv.spec_linear_ce(h, w, y)
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.spec_linear_ce_grad(h, w, y, nll, lse, g, d_hidden=h)  # the output is an input
    assert e.value.code == sv.SPEC_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        sv.spec_linear_ce_grad(h, w, y, nll, lse, g, need_hidden=False, need_weight=False)
    with pytest.raises(ValueError):
        sv.LinearCe(h, w, y).grad()
