"""Which stream a call's own tensors are allocated on."""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


def test_handles_of_streams():
    dev = torch.device("cuda", torch.cuda.current_device())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for handle, want in ((0, 0), (side.cuda_stream, side.cuda_stream), (side, side.cuda_stream)):
            with sv._alloc_on(handle, dev):
                assert torch.cuda.current_stream(dev).cuda_stream == want
    with sv._alloc_on(side.cuda_stream, dev):
        assert torch.cuda.current_stream(dev).cuda_stream == side.cuda_stream


def test_a_sampler_used_under_another_stream():
    z = torch.randn((3, 2, 5000), device="cuda")
    T = torch.full((3,), 0.7, device="cuda")
    k = torch.full((3,), 40, dtype=torch.int32, device="cuda")
    want = sv.spec_truncate(z, T, top_k=k)
    sampler = sv.Sampler(z, T, top_k=k)  # bound to the default stream
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        kept = sampler.truncate()
    torch.cuda.current_stream().synchronize()
    assert torch.equal(kept, want)
    # Its memory belongs to the stream it is written on.
    segments = [s for s in torch.cuda.memory_snapshot()
                if s["address"] <= kept.data_ptr() < s["address"] + s["total_size"]]
    assert [s["stream"] for s in segments] == [0]
