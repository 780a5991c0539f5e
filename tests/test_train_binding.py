"""The training calls' binding without a GPU: what it refuses before the library is called."""

import contextlib

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv


@pytest.fixture
def host(monkeypatch):
    """The binding on host tensors; the library's calls are recorded, not made."""
    sv.build()
    monkeypatch.setattr(sv, "_need_cuda", lambda t, name: None)
    monkeypatch.setattr(sv, "_alloc_on", lambda stream, device: contextlib.nullcontext())
    monkeypatch.setattr(sv, "_stream_on", lambda stream, device: 0)
    calls = []

    def bind(ce):
        ce._loss = lambda *a: calls.append("loss") or 0
        ce._grad = lambda *a: calls.append("grad") or 0
        return ce

    return bind, calls


def buffers(N=6, V=20, D=8):
    f = torch.zeros(N)
    return (torch.zeros(N, D, dtype=torch.bfloat16), torch.zeros(V, D, dtype=torch.bfloat16),
            torch.zeros(N, dtype=torch.int32), f)


def test_gradients_need_a_loss(host):
    bind, calls = host
    h, w, y, g = buffers()
    ce = bind(sv.LinearCe(h, w, y, g))
    with pytest.raises(ValueError, match="loss"):
        ce.grad()  # nll and lse hold nothing yet
    ce.loss()
    ce.grad()
    assert calls == ["loss", "grad"]
    # One buffer of the two is not enough; with both the caller answers for their contents.
    for kw in (dict(nll=torch.zeros(6)), dict(lse=torch.zeros(6))):
        with pytest.raises(ValueError, match="loss"):
            bind(sv.LinearCe(h, w, y, g, **kw)).grad()
    bind(sv.LinearCe(h, w, y, g, nll=torch.zeros(6), lse=torch.zeros(6))).grad()
    assert calls == ["loss", "grad", "grad"]


def test_a_loss_that_failed_is_none(host):
    bind, calls = host
    h, w, y, g = buffers()
    ce = bind(sv.LinearCe(h, w, y, g))
    ce._loss = lambda *a: sv.SPEC_ERR_CUDA
    with pytest.raises(sv.SpecVerifyError):
        ce.loss()
    with pytest.raises(ValueError, match="loss"):
        ce.grad()


@pytest.mark.parametrize("missing", ["nll", "lse", "both"])
def test_the_gradient_call_needs_both(host, monkeypatch, missing):
    h, w, y, g = buffers()
    nll = None if missing in ("nll", "both") else torch.zeros(6)
    lse = None if missing in ("lse", "both") else torch.zeros(6)
    made = []
    monkeypatch.setattr(sv, "LinearCe", lambda *a, **kw: made.append(a))
    with pytest.raises(ValueError, match="nll and lse"):
        sv.spec_linear_ce_grad(h, w, y, nll, lse, g)
    assert not made
