"""Values that are not finite, of entries whose weights are as small as single precision has no
number for: every row that sees one has no finite result in its dimension, wherever the entries
lie in a request, and the others are what they are without it."""

import math

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv
from test_gpu_paged import Batch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


@pytest.mark.parametrize("odd", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("D,G", [(128, 4), (64, 2)])
@pytest.mark.parametrize("n,t", [(1, 200), (1, 700), (1, 60000), (16, 900), (40, 3000), (90, 20000), (300, 5000)])
def test_values_of_no_weight(n, t, D, G, odd):
    b = Batch([(n, t), (1, 300)], Hk=2, G=G, D=D, P=64, seed=4)
    # The scores of one stretch of 64 entries are far above the others'.
    b.q.copy_(b.q.float().abs().to(b.q.dtype))
    peak = t // 3 // 64 * 64
    for i, size in enumerate((t, 300)):
        at = torch.arange(size, device=DEV)
        page, slot = b.table[i][at // b.P].long(), at % b.P
        high = ((at >= peak) & (at < peak + 64))[:, None, None]
        b.k[page, slot] = torch.where(high, 8.0, -8.0).to(b.k.dtype).expand(size, b.Hk, D)
    good, lse = sv.spec_paged_attention(b.q, *b.arrays(), need_lse=True)
    b.check(good, lse)
    spots = [0, 70, peak + 130, t // 2, t - n - 3, t - n, t - 1]
    for j, x in enumerate(sorted({s for s in spots if 0 <= s < t and not peak <= s < peak + 64})):
        v = b.v.clone()
        d = (7 * j) % D
        b.v[b.table[0, x // b.P].long(), x % b.P, 1, d] = odd
        out, l2 = sv.spec_paged_attention(b.q, *b.arrays(), need_lse=True)
        sees = torch.arange(t - n, t, device=DEV) >= x
        met = torch.zeros_like(out, dtype=torch.bool)
        met[:n, G:, d] = sees[:, None]
        assert torch.equal(l2, lse)
        assert bool((~torch.isfinite(out[met])).all()), (x, int(torch.isfinite(out[met]).sum()))
        assert torch.equal(out[~met], good[~met]), x
        b.v.copy_(v)


@pytest.mark.parametrize("n,t", [(1, 700), (1, 60000), (16, 900), (90, 20000)])
def test_keys_of_no_weight(n, t):
    """A NaN key far from the entries that have all the weight: NaN rows."""
    b = Batch([(n, t)], Hk=1, G=4, D=128, P=64, seed=4)
    b.q.copy_(b.q.float().abs().to(b.q.dtype))
    at = torch.arange(t, device=DEV)
    page, slot = b.table[0][at // b.P].long(), at % b.P
    peak = t // 3 // 64 * 64
    high = ((at >= peak) & (at < peak + 64))[:, None, None]
    b.k[page, slot] = torch.where(high, 8.0, -8.0).to(b.k.dtype).expand(t, 1, 128)
    k = b.k.clone()
    for x in (0, peak + 130, t // 2, t - n - 3):
        b.k.copy_(k)
        b.k[b.table[0, x // b.P].long(), x % b.P, 0, 5] = math.nan
        out, lse = sv.spec_paged_attention(b.q, *b.arrays(), need_lse=True)
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all()), x
