"""Truncated sampling and truncation against double precision."""

import math

import pytest

torch = pytest.importorskip("torch")

import round_ref as ref
import speculative_decoding_verification_58_gb300 as sv

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make(kind, B, n, V, dt, seed):
    g = gen(seed)
    z = torch.randn((B, n, V), generator=g, device=DEV)
    if kind == "zipf":
        tail = -1.1 * torch.log(torch.arange(1, V + 1, device=DEV).float())
        for b in range(B):
            z[b] += tail[torch.randperm(V, generator=g, device=DEV)]
    elif kind == "ties":
        z = torch.round(2 * z) / 2
    elif kind == "equal":
        z = torch.full_like(z, -1.5)
    elif kind == "peaked":
        z[..., V // 2] += 60.0
    elif kind == "masked":
        z[torch.rand(z.shape, generator=g, device=DEV) < 0.7] = -math.inf
        z[..., V - 1] = 0.25
    elif kind == "lowest":
        z[torch.rand(z.shape, generator=g, device=DEV) < 0.7] = torch.finfo(DT[dt]).min
        z[..., 0] = -0.25
    elif kind == "shifted":
        z += 1000.0
    elif kind == "wide":
        z *= 40.0
    return z.to(DT[dt])


def check(z, T, u, k=None, p=None, m=None, group=None):
    """Both calls against the reference, row by row; at most a few rows near a border."""
    B, n, V = z.shape
    tokens, both = sv.spec_sample(z, T, u, top_k=k, top_p=p, min_p=m, kept=torch.empty_like(z))
    only = sv.spec_sample(z, T, u, top_k=k, top_p=p, min_p=m)
    kept = sv.spec_truncate(z, T, top_k=k, top_p=p, min_p=m)
    torch.cuda.synchronize()
    assert torch.equal(tokens, only)
    assert torch.equal(both.view(torch.uint8), kept.view(torch.uint8))
    nears = 0
    for b in range(B):
        a = (float(T[b]), 0 if k is None else int(k[b]), 1.0 if p is None else float(p[b]),
             0.0 if m is None else float(m[b]))
        for i in range(n):
            keep, w, near = ref.truncate(z[b, i], *a)
            tok, near_u = ref.draw(w, float(u[b, i]))
            off = torch.where(keep, z[b, i], torch.tensor(-math.inf, device=DEV, dtype=z.dtype))
            if near or near_u:
                nears += 1
                continue
            assert torch.equal(kept[b, i], off), (b, i, a, int((kept[b, i] != off).sum()))
            assert int(tokens[b, i]) == tok, (b, i, a, float(u[b, i]), int(tokens[b, i]), tok)
    assert nears <= max(2, B * n // 20), nears


def settings(B, seed):
    g = gen(seed)

    def pick(v, dtype):
        return torch.tensor(v, dtype=dtype, device=DEV)[
            torch.randint(0, len(v), (B,), generator=g, device=DEV)]

    return (pick([0.0, 0.6, 1.0, 1.3], torch.float32),
            dict(k=pick([0, 1, 7, 50, 400, 5000], torch.int32),
                 p=pick([1.0, 0.3, 0.9, 0.99], torch.float32),
                 m=pick([0.0, 0.0, 0.05, 1e-4], torch.float32)))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["gauss", "zipf", "ties", "equal", "peaked", "masked", "lowest",
                                  "shifted", "wide"])
@pytest.mark.parametrize("V", [1, 2, 31, 257, 1000, 8192, 33333])
def test_all_settings(kind, V, dt):
    B, n = (12, 2) if V < 8000 else (8, 1)
    T, s = settings(B, V)
    u = torch.rand((B, n), generator=gen(V + 1), device=DEV)
    check(make(kind, B, n, V, dt, V + 2), T, u, **s)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["gauss", "zipf", "ties"])
def test_full_vocabulary(kind, dt):
    B, n, V = 12, 2, 151936
    T, s = settings(B, 5)
    u = torch.rand((B, n), generator=gen(6), device=DEV)
    check(make(kind, B, n, V, dt, 7), T, u, **s)
    check(make(kind, B, n, V, dt, 8), T, u)


def test_largest_vocabulary():
    V = 1 << 21
    z = make("gauss", 2, 1, V, "f32", 3)
    one = torch.ones(2, device=DEV)
    u = torch.tensor([[0.3], [0.9]], device=DEV)
    check(z, one, u)
    check(z, one, u, p=0.5 * one, k=torch.tensor([0, 100000], dtype=torch.int32, device=DEV))
    check(torch.zeros_like(z).bfloat16(), one, u, p=0.75 * one)


@pytest.mark.parametrize("T", [1.2e-38, 1e-3, 0.05, 30.0, 1e6, 3e38])
def test_extreme_temperatures(T):
    B, V = 6, 4000
    z = make("gauss", B, 1, V, "f32", 21)
    z[0] = make("ties", 1, 1, V, "f32", 2)[0]
    u = torch.rand((B, 1), generator=gen(1), device=DEV)
    t = torch.full((B,), T, device=DEV)
    check(z, t, u)
    check(z, t, u, p=torch.full((B,), 0.9, device=DEV))
    check(z, t, u, k=torch.full((B,), 33, dtype=torch.int32, device=DEV),
          p=torch.full((B,), 0.9, device=DEV), m=torch.full((B,), 0.5, device=DEV))


@pytest.mark.parametrize("p", [1e-30, 1e-6, 0.5, 0.9999, 0.999999])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_extreme_top_p(p, dt):
    B, V = 6, 20011
    T = torch.full((B,), 0.9, device=DEV)
    u = torch.rand((B, 1), generator=gen(1), device=DEV)
    for kind in ("gauss", "zipf", "equal"):
        check(make(kind, B, 1, V, dt, 4), T, u, p=torch.full((B,), p, device=DEV))


@pytest.mark.parametrize("m", [1e-30, 1e-3, 0.5, 1.0])
def test_extreme_min_p(m):
    B, V = 6, 5000
    T = torch.full((B,), 0.7, device=DEV)
    u = torch.rand((B, 1), generator=gen(1), device=DEV)
    for kind in ("gauss", "ties"):
        check(make(kind, B, 1, V, "bf16", 4), T, u, m=torch.full((B,), m, device=DEV))


@pytest.mark.parametrize("k", [1, 2, 31, 32, 33, 511, 1024, 4095, 4096, 4097, 9998, 9999, 10000, 10 ** 9])
def test_top_k_sizes(k):
    B, V = 4, 9999
    T = torch.full((B,), 1.0, device=DEV)
    u = torch.rand((B, 1), generator=gen(1), device=DEV)
    kk = torch.full((B,), k, dtype=torch.int32, device=DEV)
    for kind, dt in (("gauss", "f32"), ("gauss", "bf16"), ("ties", "f32"), ("equal", "bf16")):
        check(make(kind, B, 1, V, dt, 9), T, u, k=kk)
        check(make(kind, B, 1, V, dt, 9), T, u, k=kk, p=torch.full((B,), 0.95, device=DEV))


def test_uniform_ends():
    B, V = 2, 777
    z = make("gauss", B, 1, V, "f32", 5)
    one = torch.ones(B, device=DEV)
    for u in (0.0, 1.0 - 2.0 ** -24):
        check(z, one, torch.full((B, 1), u, device=DEV))
        check(z, one, torch.full((B, 1), u, device=DEV), k=torch.full((B,), 5, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_invalid_rows_and_settings(dt):
    B, V = 16, 3001
    z = make("gauss", B, 1, V, dt, 5)
    T = torch.full((B,), 0.8, device=DEV)
    k = torch.full((B,), 40, dtype=torch.int32, device=DEV)
    p = torch.full((B,), 0.9, device=DEV)
    m = torch.full((B,), 0.01, device=DEV)
    u = torch.full((B, 1), 0.4, device=DEV)
    z[0, 0, 100] = math.nan
    z[1, 0, V - 1] = math.inf
    z[2] = -math.inf
    T[3], T[4], T[5] = -1.0, math.nan, math.inf
    k[6] = -1
    p[7], p[8], p[9] = 0.0, 1.5, math.nan
    m[10], m[11] = -0.1, math.nan
    u[12], u[13] = 1.0, math.nan
    tokens, kept = sv.spec_sample(z, T, u, top_k=k, top_p=p, min_p=m, kept=torch.empty_like(z))
    for b in range(12):
        assert int(tokens[b]) == -1, b
        assert bool(torch.isnan(kept[b]).all()), b
    for b in (12, 13):
        assert int(tokens[b]) == -1
    for b in range(12, B):
        keep, w, near = ref.truncate(z[b, 0], 0.8000000119, 40, float(p[b]), float(m[b]))
        assert not near and torch.equal(kept[b, 0] > -math.inf, keep)
        if b > 13:
            assert int(tokens[b]) == ref.draw(w, float(u[b]))[0]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_greedy_rows(dt):
    V = 5003
    z = make("ties", 6, 1, V, dt, 5)
    z[1, 0, 7] = math.nan          # never the maximum
    z[2, 0, 4000] = z[2, 0, 9] = math.inf   # the lowest of the largest
    z[3] = -math.inf
    z[4] = math.nan
    z[5, 0] = 0.0
    z[5, 0, 17] = -0.0             # equal to 0
    T = torch.zeros(6, device=DEV)
    u = torch.full((6, 1), math.nan, device=DEV)  # not used
    bad_k = torch.full((6,), -3, dtype=torch.int32, device=DEV)  # nor these
    tokens, kept = sv.spec_sample(z, T, u, top_k=bad_k, kept=torch.empty_like(z))
    want = []
    for b in range(6):
        x = z[b, 0].double()
        x = torch.where(torch.isnan(x), -math.inf, x)
        want.append(-1 if float(x.max()) == -math.inf else int(torch.nonzero(x == x.max())[0]))
    assert tokens[:, 0].tolist() == want
    assert want[2] == 9 and want[5] == 0 and want[3] == want[4] == -1
    for b in (0, 1, 2, 5):
        only = torch.full_like(z[b, 0], -math.inf)
        only[want[b]] = z[b, 0, want[b]]
        assert torch.equal(kept[b, 0], only)
    assert bool(torch.isnan(kept[3:5]).all())


def test_negative_zero_ties():
    z = torch.zeros((1, 1, 64), device=DEV)
    z[0, 0, ::2] = -0.0
    k = torch.tensor([5], dtype=torch.int32, device=DEV)
    kept = sv.spec_truncate(z, torch.ones(1, device=DEV), top_k=k)
    assert torch.nonzero(kept[0, 0] > -math.inf)[:, 0].tolist() == [0, 1, 2, 3, 4]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("off", [1, 3, 5])
def test_off_16_byte_lines_and_in_place(dt, off):
    B, n, V = 3, 5, 10007
    T, s = settings(B, 5)
    s = {"top_k": s["k"], "top_p": s["p"], "min_p": s["m"]}
    T[:] = torch.tensor([0.7, 1.0, 0.0], device=DEV)
    u = torch.rand((B, n), generator=gen(6), device=DEV)
    z = make("zipf", B, n, V, dt, 7)
    tokens, kept = sv.spec_sample(z, T, u, kept=torch.empty_like(z), **s)
    size = B * n * V
    inbuf = torch.full((size + 16,), 7.0, dtype=z.dtype, device=DEV)
    inbuf[off:off + size] = z.flatten()
    view = inbuf[off:off + size].view(B, n, V)
    outbuf = torch.full((size + 16,), 9.0, dtype=z.dtype, device=DEV)
    out = outbuf[off + 1:off + 1 + size].view(B, n, V)
    t2, k2 = sv.spec_sample(view, T, u, kept=out, **s)
    assert torch.equal(tokens, t2) and torch.equal(kept, k2)
    assert bool((outbuf[:off + 1] == 9.0).all()) and bool((outbuf[off + 1 + size:] == 9.0).all())
    t3, k3 = sv.spec_sample(view, T, u, kept=view, **s)  # in place
    assert torch.equal(tokens, t3) and torch.equal(kept, k3)
    assert bool((inbuf[:off] == 7.0).all()) and bool((inbuf[off + size:] == 7.0).all())
    again = sv.spec_truncate(view, T, kept=view)  # truncated rows keep what they have
    assert torch.equal(again, kept)


def test_a_row_does_not_depend_on_its_batch():
    V = 40000
    z = make("gauss", 300, 1, V, "bf16", 7)
    z[77] = z[0]
    z[299] = z[0]
    T = torch.full((300,), 1.1, device=DEV)
    p = torch.full((300,), 0.97, device=DEV)
    u = torch.full((300, 1), 0.5, device=DEV)
    tokens, kept = sv.spec_sample(z, T, u, top_p=p, kept=torch.empty_like(z))
    t1, k1 = sv.spec_sample(z[:1].clone(), T[:1].clone(), u[:1].clone(), top_p=p[:1].clone(),
                            kept=torch.empty_like(z[:1]))
    for b in (0, 77, 299):
        assert int(tokens[b]) == int(t1[0]) and torch.equal(kept[b], k1[0])


def test_two_dimensional_logits_and_bound_form():
    B, V = 9, 1234
    z = make("zipf", B, 1, V, "f32", 3)[:, 0].contiguous()
    T = torch.full((B,), 0.9, device=DEV)
    u = torch.rand(B, generator=gen(2), device=DEV)
    k = torch.full((B,), 20, dtype=torch.int32, device=DEV)
    s = sv.Sampler(z, T, u, top_k=k)
    tok = s.sample().clone()
    kept = s.truncate()
    for b in range(B):
        keep, w, _ = ref.truncate(z[b], float(T[b]), 20)
        assert int(tok[b]) == ref.draw(w, float(u[b]))[0]
        assert torch.equal(kept[b] > -math.inf, keep)
    u.copy_(torch.rand(B, generator=gen(4), device=DEV))  # the same buffers, other contents
    tok = s.sample()
    for b in range(B):
        _, w, _ = ref.truncate(z[b], float(T[b]), 20)
        assert int(tok[b]) == ref.draw(w, float(u[b]))[0]


def test_graph_and_streams():
    B, n, V = 6, 4, 20000
    T, s = settings(B, 5)
    z = make("zipf", B, n, V, "bf16", 7)
    u = torch.rand((B, n), generator=gen(6), device=DEV)
    smp = sv.Sampler(z, T, u, top_k=s["k"], top_p=s["p"], min_p=s["m"], kept=torch.empty_like(z))
    tokens, kept = (t.clone() for t in smp.sample())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = sv.spec_sample(z, T, u, top_k=s["k"], top_p=s["p"], min_p=s["m"], stream=side)
    side.synchronize()
    assert torch.equal(tokens, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bound = sv.Sampler(z, T, u, top_k=s["k"], top_p=s["p"], min_p=s["m"],
                           kept=torch.empty_like(z))
        t2, k2 = bound.sample()
    for seed in (8, 9):
        z.copy_(make("zipf", B, n, V, "bf16", seed))
        graph.replay()
        want = sv.spec_sample(z, T, u, top_k=s["k"], top_p=s["p"], min_p=s["m"], kept=kept)
        torch.cuda.synchronize()
        assert torch.equal(t2, want[0]) and torch.equal(k2, want[1])


def test_past_32_bit_offsets():
    V = 151936
    rows = (1 << 32) // V + 40  # entries past 2^32, 8.6 GB
    z = torch.full((rows, V), -20.0, dtype=torch.bfloat16, device=DEV)
    at = torch.arange(rows, device=DEV) * 7919 % V
    z[torch.arange(rows, device=DEV), at] = 5.0
    T = torch.full((rows,), 0.5, device=DEV)
    u = torch.full((rows,), 0.5, device=DEV)
    k = torch.full((rows,), 3, dtype=torch.int32, device=DEV)
    tokens = sv.spec_sample(z, T, u, top_k=k)
    assert torch.equal(tokens.long(), at)
    sv.spec_truncate(z, T, top_k=k, kept=z)
    assert torch.equal((z[-64:] > -math.inf).sum(1), torch.full((64,), 3, device=DEV))


@pytest.mark.parametrize("seed", range(4))
def test_borders_of_many_flat_float_rows(seed):
    """Where the mass reaches top_p, against sums in 64 bits: entries of 10^-6 of the mass, and
    maxima whose last bits the other entries do not have."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, n, V = 16, 17, 151936
    z = torch.randn((B, n, V), generator=g, device="cuda")
    z -= 1.1 * torch.log(torch.arange(1, V + 1, device="cuda", dtype=torch.float32))
    T = 0.8 + 0.5 * torch.rand(B, generator=g, device="cuda")
    p = torch.where(torch.arange(B, device="cuda") % 2 == 0, 0.95, 0.99)
    kept = sv.spec_truncate(z, T, top_p=p) != -math.inf
    for b in range(B):
        zs, order = torch.sort(z[b], dim=1, descending=True, stable=True)
        m = torch.exp((zs.double() - zs[:, :1].double()) / T[b].double())
        upto = torch.cumsum(m, 1)
        less = upto - m - p[b].double() * upto[:, -1:]
        want = torch.zeros_like(kept[b]).scatter_(1, order, less < 0)
        unclear = torch.zeros_like(want).scatter_(1, order, less.abs() < 1e-11 * upto[:, -1:])
        assert bool(((kept[b] == want) | unclear).all())
