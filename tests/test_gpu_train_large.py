"""The training calls on buffers whose offsets pass 32 bits (needs a GB300).

Entries past 2^31 (bytes past 2^32) of each input and output are compared with double
precision; tolerances as derived in the single operators' tests.
"""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv
import train_ref as ref
import test_gpu_grad_norm as clip_test
import test_gpu_opd_grad as opd_test

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB of free device memory")
    sv.lib()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("V", [151936, 151937])  # rows in shared memory, on and off 16-byte lines
def test_mixture_gradient(V):
    B, k = 1000, 15
    assert B * k * V > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(V)
    t = torch.empty((B, k + 1, V), dtype=torch.bfloat16, device="cuda").normal_(0, 2, generator=g)
    d = torch.empty((B, k, V), dtype=torch.bfloat16, device="cuda").normal_(0, 2, generator=g)
    L = torch.randint(1, k + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    L[-1], L[-2], L[0] = k, 3, 2
    gl = torch.rand(B, generator=g, device="cuda") + 0.5
    out = torch.full_like(d, 7.0)
    sv.spec_opd_grad(t, d, L, gl, d_draft=out)
    for b in (0, 499, 942, 943, 944, B - 2, B - 1):  # 2^31 entries end in request 942
        one = slice(b, b + 1)
        opd_test.check(t[one], d[one], L[one], gl[one], out[one])
    assert not bool((out == 7.0).all(2).any())


def test_clip():
    n = 2 ** 31 + 12345
    x = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    for r in range(0, n, 1 << 28):
        x[r:r + (1 << 28)].normal_(0, 0.01)
    y = torch.randn(777, device="cuda")
    out = [torch.full_like(x, 7.0), torch.empty_like(y)]
    norm = sv.spec_clip_grad_norm([x, y], 1.0, out=out)
    want = (sum(float(c.double().square().sum()) for c in x.split(1 << 26)) +
            float(y.double().square().sum())) ** 0.5
    assert abs(float(norm) - want) <= clip_test.REL * want
    f = 1.0 / want
    for r in (0, 2 ** 30 - 5000, 2 ** 31 - 5000, n - 5000):
        a, b = x[r:r + 10000].double() * f, out[0][r:r + 10000].double()
        assert torch.all((a - b).abs() <= (2.0 ** -8 + 2 * clip_test.REL) * a.abs() + 1e-38)
    assert not bool((out[0] == 7.0).any())


def test_widest_vocabulary():
    # weight and its gradient: 2^21 rows of 1032.
    N, V, D = 40, 1 << 21, 1032
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty((V, D), dtype=torch.bfloat16, device="cuda").normal_(0, 2 / D ** 0.5, generator=g)
    h = torch.randn((N, D), generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    y[0], y[1], y[2:10] = V - 1, 2 ** 31 // D + 1, V - 2   # rows past 2^31 entries; a frequent one
    gn = torch.rand(N, generator=g, device="cuda") / N
    ce = sv.LinearCe(h, w, y, gn)
    nll, lse = ce.loss()
    dh, dw = ce.grad()
    z = torch.cat([h.double() @ w[r:r + (1 << 18)].double().t() for r in range(0, V, 1 << 18)], 1)
    rl = torch.logsumexp(z, 1)
    top = max(float((h.double().abs() @ w[r:r + (1 << 18)].double().abs().t()).max())
              for r in range(0, V, 1 << 18))
    ez = D * 2.0 ** -23 * top
    tol = ez + 2.0 ** -18 + 2.0 ** -22 * rl.abs()
    rn = rl - z.gather(1, y.long()[:, None])[:, 0]
    assert torch.all((lse.double() - rl).abs() <= tol)
    assert torch.all((nll.double() - rn).abs() <= tol + ez)
    dz = torch.exp(z - rl[:, None])
    mass = dz.clone()
    rows = torch.arange(N, device="cuda")
    dz[rows, y.long()] -= 1.0
    mass[rows, y.long()] += 1.0
    dz, mass = dz * gn.double()[:, None], mass * gn.double()[:, None]
    e = ez + 2.0 ** -18
    for r in (0, 2 ** 30 // D - 64, 2 ** 31 // D - 64, V - 256):
        part = slice(r, r + 256)
        want = dz[:, part].t() @ h.double()
        mag = dz[:, part].abs().t() @ h.double().abs()
        err = (2.0 ** -8 + (N + 8) * 2.0 ** -23) * mag + e * (mass[:, part].t() @ h.double().abs()) + \
            2.0 ** -8 * want.abs()
        assert torch.all((dw[part].double() - want).abs() <= err * 1.0001 + 1e-38)
    want = sum(dz[:, r:r + (1 << 18)] @ w[r:r + (1 << 18)].double() for r in range(0, V, 1 << 18))
    mag = sum(dz[:, r:r + (1 << 18)].abs() @ w[r:r + (1 << 18)].double().abs()
              for r in range(0, V, 1 << 18))
    other = sum(mass[:, r:r + (1 << 18)] @ w[r:r + (1 << 18)].double().abs()
                for r in range(0, V, 1 << 18))
    # (Slices of dH hold at most 65536 terms in one sum.)
    err = (2.0 ** -8 + 65544 * 2.0 ** -23) * mag + e * other + 2.0 ** -8 * want.abs()
    assert torch.all((dh.double() - want).abs() <= err * 1.0001)


def test_most_tokens_and_entries():
    # 2^18 tokens of 2^21 entries: 2^32 partials, and labels in every part.
    N, V, D = 1 << 18, 1 << 21, 8
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn((V, D), generator=g, device="cuda").to(torch.bfloat16)
    h = torch.randn((N, D), generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    y[-1], y[-2] = V - 1, -1
    ce = sv.LinearCe(h, w, y)
    nll, lse = ce.loss()
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_OK
    pick = torch.cat([torch.arange(0, N, N // 61, device="cuda"), torch.arange(N - 5, N, device="cuda")])
    rn, rl = ref.ce(h[pick], w, y[pick])
    ez = D * 2.0 ** -23 * float((h[pick].double().abs() @ w.double().abs().t()).max())
    tol = ez + 2.0 ** -18 + 2.0 ** -22 * rl.abs()
    assert torch.all((lse[pick].double() - rl).abs() <= tol)
    assert torch.all((nll[pick].double() - rn).abs() <= tol + ez)
    assert bool(torch.isfinite(lse).all()) and bool(torch.isfinite(nll).all())
