"""The draw of truncated sampling: the token that double precision gives, also for uniforms next
to the border between two entries and for rows whose mass lies far below their largest entry."""

import math

import pytest

torch = pytest.importorskip("torch")

import sample_ref as ref
import speculative_decoding_verification_58_gb300 as sv

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
FULL = 151936


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def zipf(rows, V, seed):
    g = gen(seed)
    z = torch.randn((rows, V), generator=g, device=DEV)
    tail = -1.1 * torch.log(torch.arange(1, V + 1, device=DEV).float())
    for r in range(rows):
        z[r] += tail[torch.randperm(V, generator=g, device=DEV)]
    return z


def per_row(x, n, dtype=torch.float32):
    return torch.full((n,), x, dtype=dtype, device=DEV)


def settings(n, k=0, p=1.0, m=0.0):
    return dict(top_k=per_row(k, n, torch.int32), top_p=per_row(p, n), min_p=per_row(m, n))


def check_row(z, T, u, rows, most_unclear=0.1, **kw):
    """One row [V] under every uniform of ``u`` [n], in calls of ``rows`` rows."""
    kept = sv.spec_truncate(z[None], per_row(T, 1), **settings(1, **kw))[0] > -math.inf
    w = torch.where(kept, ref.masses(z, float(per_row(T, 1))), 0.0)
    lo, hi = ref.draws(w, u)
    assert float((lo != hi).float().mean()) <= most_unclear
    for i in range(0, u.numel(), rows):
        v = u[i:i + rows]
        n = v.numel()
        tok = sv.spec_sample(z.expand(n, -1).contiguous(), per_row(T, n), v, **settings(n, **kw))
        tok = tok.long()
        off = (tok < lo[i:i + n]) | (tok > hi[i:i + n])
        assert not bool(off.any()), (int(off.sum()), n, v[off][:4].tolist(), tok[off][:4].tolist(),
                                     lo[i:i + n][off][:4].tolist())


def border_uniforms(z, T, n, seed, **kw):
    """Uniforms next to the borders between kept entries, drawn like tokens are, and evenly."""
    kept = sv.spec_truncate(z[None], per_row(T, 1), **settings(1, **kw))[0] > -math.inf
    w = torch.where(kept, ref.masses(z, float(per_row(T, 1))), 0.0)
    c = torch.cumsum(w, 0)
    g = gen(seed)
    a = torch.searchsorted(c, torch.rand(n // 2, generator=g, device=DEV).double() * c[-1])
    some = torch.nonzero(kept)[:, 0]
    b = some[torch.randint(0, some.numel(), (n - n // 2,), generator=g, device=DEV)]
    at = torch.cat([a.clamp(max=z.numel() - 1), b])
    u = ref.at_borders(c, at)
    u[::2] = ref.at_borders(c, at[::2], -1)
    return u


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["gauss", "zipf"])
@pytest.mark.parametrize("kw", [dict(), dict(k=5000), dict(m=1e-4), dict(k=5000, p=0.95)])
def test_uniforms_at_borders(kind, dt, kw):
    z = zipf(1, FULL, 3)[0] if kind == "zipf" else torch.randn(FULL, generator=gen(4), device=DEV)
    z = z.to(DT[dt])
    u = border_uniforms(z, 0.9, 1024, 5, **kw)
    check_row(z, 0.9, u, 512, **kw)
    check_row(z, 0.9, u[:48], 3, **kw)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kw", [dict(), dict(p=0.99), dict(p=0.95), dict(k=5000)])
def test_many_rows(dt, kw):
    """Rows of their own with uniforms of their own."""
    R, T = 768, 1.0
    z = zipf(R, FULL, 11).to(DT[dt])
    u = torch.rand(R, generator=gen(12), device=DEV)
    s = settings(R, **kw)
    tok = sv.spec_sample(z, per_row(T, R), u, **s).long()
    kept = sv.spec_truncate(z, per_row(T, R), **s) > -math.inf
    for r in range(R):
        lo, hi = ref.draws(torch.where(kept[r], ref.masses(z[r], T), 0.0), u[r:r + 1])
        assert int(lo) <= int(tok[r]) <= int(hi), (r, int(tok[r]), int(lo), int(hi))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("tail", ["equal", "gauss"])
@pytest.mark.parametrize("peak", [15.0, 22.5, 23.0, 30.0])
def test_one_large_entry_over_a_low_tail(peak, tail, dt):
    V = FULL
    z = torch.zeros(V, device=DEV) if tail == "equal" else \
        0.3 * torch.randn(V, generator=gen(6), device=DEV)
    z[V // 2] = peak
    z = z.to(DT[dt])
    w = ref.masses(z, 1.0)
    before, after = float(w[:V // 2].sum() / w.sum()), float(w[V // 2 + 1:].sum() / w.sum())
    g = gen(7)
    u = torch.cat([torch.rand(192, generator=g, device=DEV) * 2 * before,
                   1.0 - torch.rand(192, generator=g, device=DEV) * 2 * after,
                   1.0 - 2.0 ** -24 * torch.arange(1, 65, device=DEV),
                   torch.rand(64, generator=g, device=DEV)]).clamp(0.0, 1.0 - 2.0 ** -24)
    # (The tail's entries are 10^-7 of the mass and less: the slack may be many of them.)
    check_row(z, 1.0, u, 512, most_unclear=1.0)
    check_row(z, 1.0, u[::16].contiguous(), 2, most_unclear=1.0)
    # What the tail is given as a whole is right, to what the slack allows.
    tok = sv.spec_sample(z.expand(512, -1).contiguous(), per_row(1.0, 512), u)
    wide = ref.slack(1.0 + before + after, V, V)
    inside = (u.double() - before).abs() > 2 * wide
    inside &= (u.double() - (1.0 - after)).abs() > 2 * wide
    peaked = (u.double() > before) & (u.double() < 1.0 - after)
    assert torch.equal((tok == V // 2)[inside], peaked[inside])


def test_largest_vocabulary_peaked():
    V = 1 << 21
    z = torch.zeros(V, device=DEV, dtype=torch.bfloat16)
    z[V // 3] = 22.0
    w = ref.masses(z, 1.0)
    after = float(w[V // 3 + 1:].sum() / w.sum())
    u = 1.0 - 2 * after * torch.rand(64, generator=gen(9), device=DEV)
    check_row(z, 1.0, u.clamp(max=1.0 - 2.0 ** -24), 16, most_unclear=1.0)


def steps(V, dt, seed):
    """A thousand entries of a few values, the rest far below: what top-p keeps of such a row is
    among its largest thousand."""
    g = gen(seed)
    z = torch.full((V,), -12.0, device=DEV)
    at = torch.randperm(V, generator=g, device=DEV)[:1000]
    values = torch.tensor([5.0, 4.3, 4.1, 2.7], device=DEV)
    z[at] = values[torch.randint(0, 4, (1000,), generator=g, device=DEV)]
    z[at[0]] = 5.6
    return z.to(DT[dt])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind,T,p", [("steps", 0.7, 0.9), ("steps", 1.3, 0.9), ("zipf", 0.7, 0.5),
                                      ("zipf", 0.5, 0.8)])
def test_uniforms_at_borders_of_listed_entries(kind, T, p, dt):
    z = steps(FULL, dt, 8) if kind == "steps" else zipf(1, FULL, 3)[0].to(DT[dt])
    u = border_uniforms(z, T, 1024, 5, p=p)
    check_row(z, T, u, 512, p=p)
    check_row(z, T, u[:48], 3, p=p)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["steps", "zipf", "gauss"])
@pytest.mark.parametrize("p", [0.5, 0.9, 1.0])
def test_a_row_draws_the_same_in_every_batch(p, kind, dt):
    V = 50021
    z = steps(V, dt, 8) if kind == "steps" else (
        zipf(1, V, 3)[0] if kind == "zipf" else torch.randn(V, generator=gen(4), device=DEV)).to(DT[dt])
    u = border_uniforms(z, 0.8, 512, 5, p=p)
    want = None
    for rows in (512, 150, 37, 1):
        tok = [sv.spec_sample(z.expand(v.numel(), -1).contiguous(), per_row(0.8, v.numel()), v.contiguous(),
                              **settings(v.numel(), p=p)) for v in u[:512 if rows > 1 else 40].split(rows)]
        tok = torch.cat(tok)
        want = tok if want is None else want
        assert torch.equal(tok, want[:tok.numel()])
