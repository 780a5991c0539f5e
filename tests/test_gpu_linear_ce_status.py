"""What linear cross entropy records in its workspace, and what a timeout leaves (needs a GB300).

No wait runs out here: a loss that timed out is what its lse says, or the range-checking build
records the status on request.
"""

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv
from test_gpu_linear_ce import check_loss, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


def lost(t):
    return t.view(torch.int32) == sv.SPEC_TIMEOUT_NAN


# One piece and dH from one tile; slices of dH; several pieces.
SHAPES = [(40, 300, 64), (200, 9000, 136), (1500, 151936, 64)]


@pytest.mark.parametrize("N,V,D", SHAPES)
def test_the_gradients_keep_a_lost_loss(N, V, D):
    h, w, y, g = inputs(N, V, D, seed=21)
    ce = sv.LinearCe(h, w, y, g)
    ce.loss()
    ce.lse[N // 2:].view(torch.int32).fill_(sv.SPEC_TIMEOUT_NAN)
    ce.grad()
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_ERR_TIMEOUT
    y[0] = V  # over a bad label too
    ce.grad()
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_ERR_TIMEOUT
    # The next loss starts anew, and another NaN says nothing.
    y[0] = 0
    check_loss(h, w, y, *ce.loss())
    ce.grad()
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_OK
    ce.lse.fill_(float("nan"))
    ce.grad()
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_OK


def run_debug(code):
    text = """
import sys
sys.path.insert(0, {tests!r}); sys.path.insert(0, {root!r})
import torch
import speculative_decoding_verification_58_gb300 as sv
import test_gpu_linear_ce_status as t
assert sv.spec_debug_build()
""".format(tests=os.path.dirname(os.path.abspath(__file__)),
           root=os.path.dirname(os.path.dirname(os.path.abspath(__file__)))) + code + "\nprint('done')\n"
    r = subprocess.run([sys.executable, "-c", text], env=dict(os.environ, SPEC_VERIFY_DEBUG="1"),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "done" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]


def test_a_loss_that_timed_out():
    run_debug("""
for N, V, D in t.SHAPES:
    h, w, y, g = t.inputs(N, V, D, seed=22)
    ce = sv.LinearCe(h, w, y, g)
    sv.spec_debug_inject(sv.SPEC_ERR_TIMEOUT)
    nll, lse = ce.loss()
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_ERR_TIMEOUT
    assert bool(t.lost(nll).all()) and bool(t.lost(lse).all())
    sv.spec_debug_inject(sv.SPEC_OK)
    ce.grad()
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_ERR_TIMEOUT
    t.check_loss(h, w, y, *ce.loss())
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_OK
""")


def test_the_release_build_injects_nothing():
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.spec_debug_inject(sv.SPEC_ERR_TIMEOUT)
    assert e.value.code == sv.SPEC_ERR_UNSUPPORTED


@pytest.mark.parametrize("N,V,D", SHAPES)
def test_no_gradients_of_a_lost_loss(N, V, D):
    h, w, y, g = inputs(N, V, D, seed=23)
    ce = sv.LinearCe(h, w, y, g)
    ce.loss()
    want = [t.clone() for t in ce.grad()]
    nll, lse = ce.nll.clone(), ce.lse.clone()
    lse[y < 0] = 0.0  # (not read for a token without a label)
    # An ordinary NaN spoils what it enters: every entry of the token's dZ but the
    # label's, which is exp(-nll) - 1.
    last = int((y >= 0).nonzero()[-1])
    ce.lse[last] = float("nan")
    dh, dw = ce.grad()
    assert torch.isnan(dh).all(1).nonzero().tolist() == [[last]]
    assert int(torch.isnan(dh).any(1).sum()) == 1
    assert (~torch.isnan(dw)).any(1).nonzero().tolist() == [[int(y[last])]]
    lse[0].view(torch.int32).fill_(sv.SPEC_TIMEOUT_NAN)
    for kw in (dict(), dict(need_hidden=False), dict(need_weight=False)):
        for t in sv.spec_linear_ce_grad(h, w, y, nll, lse, g, **kw):
            assert t is None or bool(torch.isnan(t).all())
    ce.loss()
    assert all(torch.equal(a, b) for a, b in zip(want, ce.grad()))


def test_gradients_that_timed_out():
    run_debug("""
for N, V, D in t.SHAPES:
    h, w, y, g = t.inputs(N, V, D, seed=24)
    ce = sv.LinearCe(h, w, y, g)
    ce.loss()
    want = [x.clone() for x in ce.grad()]
    sv.spec_debug_inject(sv.SPEC_ERR_TIMEOUT)
    for x in ce.grad():
        assert bool(torch.isnan(x).all())
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_ERR_TIMEOUT
    sv.spec_debug_inject(sv.SPEC_OK)
    for x, z in zip(ce.grad(), want):
        assert torch.equal(x, z)
    assert sv.spec_verify_device_status(ce.workspace) == sv.SPEC_OK
assert sv.spec_debug_checks()[0] == 0
""")
