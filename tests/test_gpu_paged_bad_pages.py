"""A page outside the cache makes the rows NaN that see an entry of it, and no others."""

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


@pytest.mark.parametrize("first_page", [0.5, math.nan, math.inf])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 3), (True, 60), (False, 0)])
@pytest.mark.parametrize("D,G,P", [(128, 4, 16), (64, 2, 8), (128, 1, 64), (64, 8, 256)])
def test_rows_that_do_not_see_it(D, G, P, causal, window, first_page):
    sizes = [(17, 300), (5, 5), (1, 77), (40, 400), (100, 300), (300, 520), (2, 1300)]
    b = Batch(sizes, Hk=2, G=G, D=D, P=P, seed=11)
    # The cache's first page belongs to nobody, and may hold anything.
    for name in ("k", "v"):
        c = getattr(b, name)
        setattr(b, name, torch.cat([torch.full_like(c[:1], first_page), c]))
    b.table = torch.where((b.table >= 0) & (b.table < 1 << 20), b.table + 1, b.table)
    kw = dict(causal=causal, window=window, need_lse=True)
    ws = torch.zeros(int(sv.lib().spec_paged_attention_workspace_bytes(b.rows, b.H, b.Hk, b.D)),
                     dtype=torch.uint8, device=DEV)
    good, good_l = sv.spec_paged_attention(b.q, *b.arrays(), workspace=ws, **kw)
    assert sv.spec_verify_device_status(ws) == sv.SPEC_OK
    b.check(good, good_l, causal, window)
    whole = b.table.clone()
    for where in ("last", "of the first new token", "before it", "first"):
        b.table.copy_(whole)
        bad = []
        for i, (n, t) in enumerate(sizes):
            at = {"last": t - 1, "of the first new token": t - n, "before it": max(0, t - n - P),
                  "first": 0}[where]
            b.table[i, at // P] = (-1, b.k.shape[0], 2 ** 31 - 1)[i % 3]
            pos = torch.arange(t - n, t, device=DEV)[:, None]
            j = torch.arange(at // P * P, min(t, at // P * P + P), device=DEV)[None, :]
            sees = torch.ones((n, j.numel()), dtype=torch.bool, device=DEV)
            if causal:
                sees = j <= pos
                if window:
                    sees &= j > pos - window
            bad.append(sees.any(1))
        bad = torch.cat(bad)
        out, lse = sv.spec_paged_attention(b.q, *b.arrays(), workspace=ws, **kw)
        assert sv.spec_verify_device_status(ws) == (sv.SPEC_ERR_BAD_INPUT if bool(bad.any())
                                                    else sv.SPEC_OK)
        assert bool(torch.isnan(out[bad]).all()) and bool(torch.isnan(lse[bad]).all()), where
        assert torch.equal(out[~bad], good[~bad]) and torch.equal(lse[~bad], good_l[~bad]), where
