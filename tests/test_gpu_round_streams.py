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
