"""What top-p keeps, for shares next to the sums of a row's largest entries: what double precision
keeps, on rows whose masses' errors average out and on rows where they do not."""

import math

import pytest

torch = pytest.importorskip("torch")

import sample_ref as ref
import speculative_decoding_verification_58_gb300 as sv
from test_gpu_sample_draw import gen, per_row, steps, zipf

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
FULL = 151936


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


def check(z, T, p, rows, most_unclear=0.1):
    """One row [V] under every share of ``p`` [n], in calls of ``rows`` rows."""
    V, n = z.numel(), p.numel()
    order = torch.argsort(-z.double(), stable=True)
    place = torch.empty_like(order).scatter_(0, order, torch.arange(V, device=DEV))
    lo, hi = ref.counts(ref.masses(z, float(per_row(T, 1)))[order], p)
    assert float((lo != hi).float().mean()) <= most_unclear
    for i in range(0, n, rows):
        q = p[i:i + rows].contiguous()
        m = q.numel()
        kept = sv.spec_truncate(z.expand(m, -1).contiguous(), per_row(T, m), top_p=q) > -math.inf
        count = kept.sum(1)
        off = (count < lo[i:i + m]) | (count > hi[i:i + m])
        assert not bool(off.any()), (int(off.sum()), m, q[off][:4].tolist(), count[off][:4].tolist(),
                                     lo[i:i + m][off][:4].tolist())
        assert torch.equal(kept, place[None] < count[:, None])


def border_shares(z, T, n, seed, largest=None):
    """Shares next to sums of the largest entries, spread evenly over the sums and over the
    entries (the ``largest`` ones)."""
    w = torch.sort(ref.masses(z, float(per_row(T, 1))), descending=True).values
    c = torch.cumsum(w, 0)
    g = gen(seed)
    top = w.numel() if largest is None else largest
    a = torch.searchsorted(c, torch.rand(n // 2, generator=g, device=DEV).double() * c[top - 1])
    b = torch.randint(0, top, (n - n // 2,), generator=g, device=DEV)
    at = torch.cat([a.clamp(max=top - 1), b])
    p = ref.at_borders(c, at)
    p[1::3] = ref.at_borders(c, at[1::3], 1)
    p[2::3] = ref.at_borders(c, at[2::3], -1)
    return p


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind,T", [("gauss", 0.9), ("zipf", 0.9), ("zipf", 0.7), ("steps", 1.0)])
def test_shares_at_borders(kind, T, dt):
    z = {"gauss": lambda: torch.randn(FULL, generator=gen(4), device=DEV),
         "zipf": lambda: zipf(1, FULL, 3)[0], "steps": lambda: steps(FULL, dt, 8)}[kind]().to(DT[dt])
    # (Where entries are as small as the masses' units allow, either side may be taken.)
    p = border_shares(z, T, 512, 5, largest={"steps": 1000}.get(kind, 20000 if T < 0.9 else FULL))
    check(z, T, p, 256, most_unclear=0.5)
    check(z, T, p[:48], 2, most_unclear=0.5)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("heavy", [2, 3, 5, 10])
def test_a_few_heavy_entries(heavy, dt):
    g = gen(heavy)
    for T in (0.7, 1.0):
        z = torch.randn(FULL, generator=g, device=DEV) - 14.0
        z[torch.randperm(FULL, generator=g, device=DEV)[:heavy]] = \
            0.5 * torch.randn(heavy, generator=g, device=DEV)
        z = z.to(DT[dt])
        p = border_shares(z, T, 384, 5, largest=heavy)
        check(z, T, p, 384, most_unclear=0.5)
        check(z, T, p[:32], 2, most_unclear=0.5)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("low", [0.3, 2.0, 7.0])
def test_rows_of_two_values(low, dt):
    """Rows of 32 to 2000 entries at one value and the rest at another, each with a share whose
    border is among the lower ones: thousands of equal entries have one error."""
    R, V = 512, FULL
    g = gen(int(10 * low))
    T = 0.4 + torch.rand(R, generator=g, device=DEV)
    top = (2.0 * torch.randn(R, generator=g, device=DEV)).to(DT[dt])
    bottom = (top.float() - low * T * (0.5 + torch.rand(R, generator=g, device=DEV))).to(DT[dt])
    many = torch.randint(32, 2000, (R,), generator=g, device=DEV)
    w = torch.exp((bottom.double() - top.double()) / T.double())
    total = many + (V - many) * w
    k = (torch.rand(R, generator=g, device=DEV) * (V - many)).long()  # of the lower ones
    p = ((many + k * w) / total).float().clamp(2.0 ** -24, 1.0 - 2.0 ** -24)
    z = bottom[:, None].expand(R, V).contiguous()
    for r in range(R):
        z[r, torch.randperm(V, generator=g, device=DEV)[:int(many[r])]] = top[r]
    kept = sv.spec_truncate(z, T, top_p=p) > -math.inf
    count = kept.sum(1)
    need = (p.double() * total - many) / w
    s = ref.slack(total, V, V) / w
    lo, hi = many + torch.ceil(need - s).clamp(min=0), many + torch.ceil(need + s)
    assert float((lo != hi).float().mean()) <= 0.1
    off = (count < lo) | (count > hi)
    assert not bool(off.any()), (int(off.sum()), count[off][:4].tolist(), lo[off][:4].tolist())
    for r in range(0, R, 16):
        order = torch.argsort(-z[r].double(), stable=True)
        assert bool(kept[r][order[:int(count[r])]].all())


def test_rows_do_not_depend_on_their_batch():
    for dt in ("f32", "bf16"):
        z = zipf(1, 50021, 3)[0].to(DT[dt])
        p = border_shares(z, 0.8, 300, 5)
        want = sv.spec_truncate(z.expand(300, -1).contiguous(), per_row(0.8, 300), top_p=p)
        for rows in (37, 1):
            for i in range(0, 37 if rows > 1 else 24, rows):
                q = p[i:i + rows].contiguous()
                got = sv.spec_truncate(z.expand(rows, -1).contiguous(), per_row(0.8, rows), top_p=q)
                assert torch.equal(got, want[i:i + rows])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_far_from_zero_at_low_temperatures(dt):
    """Logits whose quotients by the temperature are too large for the quick masses."""
    V = 30011
    z = (0.02 * torch.randn(V, generator=gen(2), device=DEV) + 700.0) if dt == "f32" else \
        700.0 + 4.0 * torch.randint(0, 40, (V,), generator=gen(2), device=DEV)
    z = z.to(DT[dt])
    T = 0.02 if dt == "f32" else 40.0
    check(z, T, border_shares(z, T, 64, 5), 64, most_unclear=0.5)
