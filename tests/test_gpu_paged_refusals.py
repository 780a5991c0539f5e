"""Host memory where the paged cache's calls want device memory."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv
from test_gpu_paged import BF, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


@pytest.mark.parametrize("pinned", [True, False])
def test_host_memory(pinned):
    b = Batch([(3, 40), (1, 20)])
    new = torch.ones((b.rows, b.Hk, b.D), dtype=BF, device="cuda")
    bound = sv.PagedCache(*b.arrays(), k_new=new, v_new=new, q=b.q)
    c = bound._c
    host = torch.zeros(b.k.numel() + 64, dtype=BF)
    host = host.pin_memory() if pinned else host
    at = (host.data_ptr() + 255) // 256 * 256
    k = c.k_cache
    c.k_cache = at
    row = b.Hk * b.D
    assert sv.lib().spec_kv_append(ctypes.byref(c), 1, new.data_ptr(), new.data_ptr(), b.rows, row, row,
                                   None) == sv.SPEC_ERR_INVALID_ARG
    c.k_cache = k
    ws = torch.zeros(1 << 26, dtype=torch.uint8)
    ws = ws.pin_memory() if pinned else ws
    at = (ws.data_ptr() + 255) // 256 * 256
    args = list(bound._attend_args)
    args[-3], args[-2] = at, (1 << 26) - 256
    assert sv.lib().spec_paged_attention(*args) == sv.SPEC_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert bool((host == 0).all()) and bool((ws == 0).all())
    bound.append()
    b.check(bound.attend(), None)
