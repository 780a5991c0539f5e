"""Drafter-training entry points without a GPU: argument checks that return before any CUDA
call, and the tests' double-precision gradients against differences."""

import ctypes

import pytest

import speculative_decoding_verification_58_gb300 as sv


@pytest.fixture(scope="module")
def lib():
    sv.build()
    return sv.lib()


def test_linear_ce_sizes(lib):
    f, g = lib.spec_linear_ce_workspace_bytes, lib.spec_linear_ce_grad_workspace_bytes
    for ws in (f, g):
        assert ws(1, 1, 8) > 0 and ws(2048, 151936, 4096) % 256 == 0
        assert ws(0, 10, 8) == ws(10, 0, 8) == ws(10, 10, 0) == 0
        assert ws(1, 10, 12) == 0                        # width not a multiple of 8
        assert ws((1 << 18) + 1, 10, 8) == 0
        assert ws(1, (1 << 21) + 1, 8) == 0
        assert ws(1, 10, (1 << 15) + 8) == 0


def test_linear_ce_host_checks(lib):
    A = 1 << 20  # addresses that are never read

    def loss(h=A, w=2 * A, dt=1, y=3 * A, N=4, V=32, D=16, nll=4 * A, lse=5 * A, ws=6 * A, n=1 << 20):
        return lib.spec_linear_ce(h, w, dt, y, N, V, D, nll, lse, ws, n, None)

    bad, uns, wsp = sv.SPEC_ERR_INVALID_ARG, sv.SPEC_ERR_UNSUPPORTED, sv.SPEC_ERR_WORKSPACE
    for kw in (dict(N=0), dict(V=0), dict(D=0), dict(h=None), dict(w=None), dict(y=None),
               dict(nll=None), dict(lse=None), dict(dt=7), dict(h=A + 8), dict(w=2 * A + 2),
               dict(y=3 * A + 1), dict(nll=A), dict(lse=2 * A + 16), dict(lse=4 * A + 4)):
        assert loss(**kw) == bad, kw
    for kw in (dict(dt=0), dict(D=12), dict(V=(1 << 21) + 1), dict(N=(1 << 18) + 1)):
        assert loss(**kw) == uns, kw
    for kw in (dict(ws=None), dict(ws=6 * A + 16), dict(n=16)):
        assert loss(**kw) == wsp, kw

    def grad(h=A, w=2 * A, dt=1, y=3 * A, nll=9 * A, lse=4 * A, g=5 * A, N=4, V=32, D=16, dh=7 * A, dw=8 * A,
             ws=6 * A, n=1 << 20):
        return lib.spec_linear_ce_grad(h, w, dt, y, nll, lse, g, N, V, D, dh, dw, ws, n, None)

    for kw in (dict(N=0), dict(g=None), dict(lse=None), dict(nll=None), dict(dh=None, dw=None), dict(dh=A),
               dict(dw=2 * A), dict(dh=8 * A), dict(dw=8 * A + 2), dict(dt=-1), dict(dw=4 * A), dict(dh=9 * A)):
        assert grad(**kw) == bad, kw
    assert grad(dt=0) == uns and grad(D=20) == uns
    assert grad(n=100) == wsp


def test_opd_grad_host_checks(lib):
    A = 1 << 20

    def f(t=A, d=2 * A, dt=0, L=3 * A, g=4 * A, B=2, k=3, V=64, delta=0.01, alpha=0.8, out=5 * A):
        return lib.spec_opd_grad(t, d, dt, L, g, B, k, V, delta, alpha, out, None)

    for kw in (dict(B=0), dict(k=0), dict(V=0), dict(dt=2), dict(delta=0.0), dict(alpha=2.0),
               dict(delta=float("nan")), dict(t=None), dict(d=None), dict(L=None), dict(g=None),
               dict(out=None), dict(t=A + 2), dict(out=5 * A + 1), dict(out=2 * A + 8),
               dict(out=A + 64), dict(out=3 * A)):
        assert f(**kw) == sv.SPEC_ERR_INVALID_ARG, kw
    assert f(k=32) == sv.SPEC_ERR_UNSUPPORTED


def test_grad_norm_host_checks(lib):
    A = 1 << 20
    assert lib.spec_grad_norm_workspace_bytes(0) == 0
    assert lib.spec_grad_norm_workspace_bytes((1 << 20) + 1) == 0
    assert 0 < lib.spec_grad_norm_workspace_bytes(1) <= lib.spec_grad_norm_workspace_bytes(2000)

    def f(grads=(A, 2 * A), outs=None, sizes=(10, 20), dts=(0, 1), max_norm=1.0, norm=3 * A,
          ws=4 * A, n=1 << 22, count=None, clip=True):
        m = len(grads)
        vp = lambda v: (ctypes.c_void_p * m)(*v)  # noqa: E731
        a = (vp(grads),) + ((None if outs is None else vp(outs),) if clip else ())
        a += ((ctypes.c_longlong * m)(*sizes), (ctypes.c_int * m)(*dts), m if count is None else count)
        a += (max_norm,) if clip else ()
        return (lib.spec_clip_grad_norm if clip else lib.spec_grad_norm)(*a, norm, ws, n, None)

    bad = sv.SPEC_ERR_INVALID_ARG
    for kw in (dict(count=0), dict(count=-1), dict(sizes=(10, -1)), dict(dts=(0, 5)),
               dict(grads=(A, None)), dict(grads=(A + 2, 2 * A)), dict(grads=(A, 2 * A + 1)),
               dict(norm=None), dict(norm=3 * A + 2), dict(norm=A), dict(max_norm=0.0),
               dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=float("inf")),
               dict(grads=(A, A)), dict(grads=(A, A + 36)), dict(outs=(5 * A, 5 * A)),
               dict(outs=(A + 4, 5 * A)), dict(outs=(2 * A, A)), dict(outs=(5 * A, None)),
               dict(outs=(5 * A, 3 * A))):
        assert f(**kw) == bad, kw
    assert f(sizes=(1 << 41, 20)) == sv.SPEC_ERR_UNSUPPORTED
    for kw in (dict(ws=None), dict(ws=4 * A + 8), dict(n=64), dict(outs=(A, 5 * A), n=64),
               dict(grads=(A, A), clip=False, n=64)):
        assert f(**kw) == sv.SPEC_ERR_WORKSPACE, kw


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    h, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(9, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sv.spec_linear_ce(h, w, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.spec_grad_norm([torch.zeros(5)])
    with pytest.raises(ValueError):
        sv.spec_opd_grad(torch.zeros(1, 3, 8), torch.zeros(1, 2, 8), torch.ones(1, dtype=torch.int32),
                         torch.ones(1))


def test_reference_gradients_against_differences():
    torch = pytest.importorskip("torch")
    import train_ref as ref
    gen = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    # Linear cross entropy.
    h, w, y, g = rnd(5, 8), rnd(11, 8), torch.tensor([0, 10, -1, 4, 4]), rnd(5)
    dh, dw, _, _ = ref.ce_grad(h, w, y, g)
    for x, grad in ((h, dh), (w, dw)):
        for _ in range(4):
            d, e = rnd(*x.shape), 1e-5
            x0 = x.clone()
            f = []
            for s in (1, -1):
                x.copy_(x0 + s * e * d)
                f.append(float((ref.ce(h, w, y)[0] * g).sum()))
            x.copy_(x0)
            assert abs((f[0] - f[1]) / (2 * e) - float((grad * d).sum())) < 1e-7
    # Mixture loss, with a clip that holds some entries.
    zt, zd, L = 2 * rnd(3, 4, 20), 2 * rnd(3, 3, 20), torch.tensor([3, 1, 2])
    gl = rnd(3)
    for delta, alpha in ((0.01, 0.8), (1e9, 0.3), (0.05, 0.0)):
        out = ref.opd_grad(zt, zd, L, gl, delta, alpha)[0]
        assert not ref.opd_grad(zt, zd, L, gl, delta, alpha, flip=1e-4)[3].any()
        for _ in range(4):
            d, e = rnd(*zd.shape), 1e-6
            f = [float((ref.opd_loss(zt, zd + s * e * d, L, delta, alpha) * gl).sum()) for s in (1, -1)]
            assert abs((f[0] - f[1]) / (2 * e) - float((out * d).sum())) < 1e-6
    assert torch.all(out[1, 1:] == 0)
