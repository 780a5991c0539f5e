"""Global gradient norm and clipping on the GPU against double precision (needs a GB300).

Tolerances.  A thread's share of at most 64 squares is summed in single
precision (64 2^-24 relative, all terms positive), everything above in
float-float, and the norm is the root of that, rounded once: 2^-18 of the norm
covers it.  A scaled entry is off by that of the scale, one rounding in single
precision and half a step of its type.
"""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv
import train_ref as ref

pytestmark = pytest.mark.gpu

REL = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


def tensors(sizes, seed=0, scale=0.1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(
        torch.bfloat16 if i % 3 else torch.float32) for i, n in enumerate(sizes)]


def check(before, after, norm, max_norm):
    want = ref.norm(before)
    assert abs(float(norm) - want) <= REL * want + 1e-44
    f = min(1.0, max_norm / want) if want > 0 else 1.0
    for a, b in zip(before, after):
        t = a.double() * f
        half = torch.finfo(a.dtype).eps / 2
        tiny = torch.finfo(a.dtype).tiny * torch.finfo(a.dtype).eps  # a step of a subnormal
        assert torch.all((b.double() - t).abs() <= (half + 2 * REL) * t.abs() + tiny)


SIZES = [
    [1], [7], [8], [0, 5, 0], [3, 1, 2, 17, 1000],
    [16383, 16384, 16385, 8191, 8192, 8193], [100003, 1, 65536, 33],
    [1 << 22, 12345], [257] * 600, [1 + (i * 37) % 500 for i in range(1100)],
]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("max_norm", [0.01, 1e6])
def test_norm_and_clip(sizes, max_norm):
    grads = tensors(sizes, seed=len(sizes))
    before = [t.clone() for t in grads]
    n0 = sv.spec_grad_norm(grads)
    out = [torch.full_like(t, 9.0) for t in grads]
    n1 = sv.spec_clip_grad_norm(grads, max_norm, out=out)
    for a, b in zip(grads, before):
        assert torch.equal(a, b)
    check(before, out, n1, max_norm)
    n2 = sv.spec_clip_grad_norm(grads, max_norm)
    check(before, grads, n2, max_norm)
    assert torch.equal(n0, n1) and torch.equal(n1, n2)
    for a, b in zip(grads, out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shift_in,shift_out", [(1, 1), (3, 3), (1, 2), (0, 1), (5, 0)])
def test_unaligned_views(shift_in, shift_out):
    # Views that start off a 16-byte line, alike or not; neighbours stay as they are.
    for dt in (torch.bfloat16, torch.float32):
        for n in (1, 2, 15, 40000):
            base = torch.randn(n + 16, device="cuda").to(dt)
            dst = torch.full((n + 16,), 7.0, dtype=dt, device="cuda")
            x, y = base[shift_in:shift_in + n], dst[shift_out:shift_out + n]
            norm = sv.spec_clip_grad_norm([x], 0.25, out=[y])
            check([x], [y], norm, 0.25)
            assert torch.all(dst[:shift_out] == 7) and torch.all(dst[shift_out + n:] == 7)


@pytest.mark.parametrize("value", [1e-45, 1e-38, 1e-30, 1e-20, 1e15, 1e25, 3e38])
def test_the_whole_range_of_single_precision(value):
    a = torch.full((5000,), value, device="cuda")
    b = torch.full((3,), value, device="cuda").to(torch.bfloat16)
    out = [torch.empty_like(a), torch.empty_like(b)]
    norm = sv.spec_clip_grad_norm([a, b], 1.0, out=out)
    want = ref.norm([a, b])
    if want > 3.4028235e38:
        assert torch.isinf(norm).all()
        f = 1.0 / want
        assert torch.all((out[0].double() - value * f).abs() <= 1e-5 * value * f)
    else:
        check([a, b], out, norm, 1.0)


def test_mixed_magnitudes():
    a = torch.tensor([1e30, 1e-30, 3.0, -0.0, 0.0], device="cuda")
    b = torch.full((100,), 1e-40, device="cuda")
    c = torch.full((70000,), 2e-25, device="cuda").to(torch.bfloat16)
    for group in ([a, b, c], [b, c], [b], [c]):
        out = [torch.empty_like(t) for t in group]
        check(group, out, sv.spec_clip_grad_norm(group, 5.0, out=out), 5.0)


def test_all_zero():
    z = [torch.zeros(1000, device="cuda"), torch.zeros(40000, dtype=torch.bfloat16, device="cuda")]
    assert float(sv.spec_clip_grad_norm(z, 1.0)) == 0.0
    assert all(torch.all(t == 0) for t in z)
    empty = [torch.zeros(0, device="cuda")]
    assert float(sv.spec_grad_norm(empty)) == 0.0
    assert float(sv.spec_clip_grad_norm(empty, 1.0)) == 0.0


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_not_finite(bad, dtype):
    for at in (0, 20000, 49999):
        a = torch.randn(50000, device="cuda").to(dtype)
        a[at] = bad
        b = torch.randn(77, device="cuda")
        a0, b0 = a.clone(), b.clone()
        norm = float(sv.spec_clip_grad_norm([a, b], 1.0))
        assert norm != norm if bad != bad else norm == float("inf")
        assert torch.equal(a.view(torch.int32 if dtype == torch.float32 else torch.int16),
                           a0.view(torch.int32 if dtype == torch.float32 else torch.int16))
        assert torch.equal(b, b0)


def test_exactly_at_the_largest_norm():
    a = torch.zeros(10, device="cuda")
    a[0], a[1] = 3.0, 4.0
    norm = sv.spec_clip_grad_norm([a], 5.0)
    assert float(norm) == 5.0 and float(a[0]) == 3.0 and float(a[1]) == 4.0


def test_bound_clipper_graph_and_streams():
    grads = tensors([5000, 333, 70001], seed=5)
    out = [torch.empty_like(t) for t in grads]
    c = sv.GradClipper(grads, 0.5, out=out)
    check(grads, out, c(), 0.5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out2 = [torch.empty_like(t) for t in grads]
    n2 = sv.spec_clip_grad_norm(grads, 0.5, out=out2, stream=s)
    s.synchronize()
    assert torch.equal(n2, c.norm) and all(torch.equal(a, b) for a, b in zip(out, out2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = sv.GradClipper(grads, 0.5, out=out, norm=c.norm, workspace=c.workspace)
        cap()
    for t in grads:
        t.mul_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    check(grads, out, c.norm, 0.5)
    # Called again and again without a wait in between: the same bits.
    first = [t.clone() for t in out]
    for _ in range(20):
        c()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_refusals():
    a, b = torch.randn(64, device="cuda"), torch.randn(64, device="cuda")
    for call in (lambda: sv.spec_clip_grad_norm([a, a], 1.0),            # scaled twice
                 lambda: sv.spec_clip_grad_norm([a[:40], a[30:]], 1.0),  # overlapping
                 lambda: sv.spec_clip_grad_norm([a, b], 1.0, out=[b, a]),
                 lambda: sv.spec_clip_grad_norm([a[:32]], 1.0, out=[a[8:40]]),
                 lambda: sv.spec_clip_grad_norm([a], 0.0),
                 lambda: sv.spec_clip_grad_norm([a], float("inf")),
                 lambda: sv.spec_clip_grad_norm([a], float("nan")),
                 lambda: sv.spec_clip_grad_norm([a], 1.0, norm=a[:1])):
        with pytest.raises(sv.SpecVerifyError) as e:
            call()
        assert e.value.code == sv.SPEC_ERR_INVALID_ARG
    # Reading one tensor twice is fine where nothing is written to it.
    assert abs(float(sv.spec_grad_norm([a, a])) - ref.norm([a, a])) <= REL * ref.norm([a, a])
    with pytest.raises(ValueError):
        sv.spec_grad_norm([])
    with pytest.raises(TypeError):
        sv.spec_grad_norm([a.double()])
    with pytest.raises(ValueError):
        sv.spec_grad_norm([a.reshape(8, 8)[:, :4]])
    with pytest.raises(ValueError):
        sv.spec_clip_grad_norm([a], 1.0, out=[a, b])
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.spec_grad_norm([a], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.code == sv.SPEC_ERR_WORKSPACE
