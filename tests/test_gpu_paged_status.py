"""What paged attention records and leaves after a timeout, and the range checks of sampling and of
the paged cache, in the range-checking build (a child process; no wait runs out)."""

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def child() -> None:
    import speculative_decoding_verification_58_gb300 as sv
    from test_gpu_paged import Batch
    import test_gpu_sample as ts

    assert sv.spec_debug_build()
    sv.spec_debug_checks(reset=True)
    b = Batch([(3, 40), (17, 300), (0, 9), (200, 500)])
    ws = torch.zeros(int(sv.lib().spec_paged_attention_workspace_bytes(b.rows, b.H, b.Hk, b.D)),
                     dtype=torch.uint8, device="cuda")

    def run():
        out = sv.spec_paged_attention(b.q, *b.arrays(), need_lse=True, workspace=ws)
        torch.cuda.synchronize()
        return out

    b.check(*run())
    sv.spec_debug_inject(sv.SPEC_ERR_TIMEOUT)
    out, lse = run()
    assert sv.spec_verify_device_status(ws) == sv.SPEC_ERR_TIMEOUT
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
    sv.spec_debug_inject(sv.SPEC_OK)
    b.check(*run())
    assert sv.spec_verify_device_status(ws) == sv.SPEC_OK
    new = torch.randn((b.rows, b.Hk, b.D), device="cuda").to(torch.bfloat16)
    sv.spec_kv_append(new, new, *b.arrays())
    b.run(False)
    for kind, V, dt in (("zipf", 5003, "bf16"), ("ties", 777, "f32"), ("gauss", 40000, "bf16")):
        T, s = ts.settings(8, 3)
        u = torch.rand((8, 2), generator=ts.gen(4), device="cuda")
        ts.check(ts.make(kind, 8, 2, V, dt, 5), T, u, **s)
    torch.cuda.synchronize()
    failures, site = sv.spec_debug_checks()
    print(f"range checks failed: {failures} (first site {site})")


def test_timeouts_and_range_checks():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    env = dict(os.environ, SPEC_VERIFY_DEBUG="1",
               PYTHONPATH=os.pathsep.join([os.path.dirname(HERE), HERE, os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", "import test_gpu_paged_status as t; t.child()"], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "range checks failed: 0" in r.stdout, r.stdout[-2000:]


def test_a_release_build_refuses_to_inject():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_58_gb300 as sv
    if sv.spec_debug_build():
        pytest.skip("the range-checking build is loaded")
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_debug_inject(sv.SPEC_ERR_TIMEOUT)
