"""Further refusals of the paged cache's and sampling's calls, before any CUDA call (no GPU needed)."""

import contextlib
import ctypes

import pytest

import speculative_decoding_verification_58_gb300 as sv
from test_round_abi import A, BAD, WSP, cache, lib  # noqa: F401 (a fixture)


def attend(lib, q=6 * A, rows=5, H=4, out=7 * A, lse=8 * A, w=9 * A, n=1 << 40, window=0, **kw):
    c = cache(**kw)
    return lib.spec_paged_attention(ctypes.byref(c), 1, q, rows, H, 256, 1, window, 0.1, out, lse, w, n,
                                    None)


def test_a_workspace_inside_another_argument(lib):
    size = int(lib.spec_paged_attention_workspace_bytes(5, 4, 2, 64))
    assert size % 256 == 0
    # What an argument's last byte is in, and what ends behind its first.
    for at, n in ((6 * A, 5 * 4 * 64 * 2), (7 * A, 5 * 4 * 64 * 2), (8 * A, 5 * 4 * 4), (3 * A, 3 * 4 * 4),
                  (4 * A, 16), (5 * A, 12), (A, 10 * 16 * 2 * 64 * 2), (2 * A, 10 * 16 * 2 * 64 * 2)):
        for w in (at, (at + n - 1) // 256 * 256, at - size + 256):
            assert attend(lib, w=w) == BAD, (hex(at), hex(w))
    assert attend(lib, w=7 * A, n=size - 1) == WSP


def test_one_cache_as_keys_and_values(lib):
    def append(**kw):
        c = cache(**kw)
        return lib.spec_kv_append(ctypes.byref(c), 1, 6 * A, 7 * A, 5, 128, 128, None)

    assert append(v_cache=A) == BAD and append(v_cache=A + 64) == BAD and append(k_cache=2 * A + 112) == BAD
    # Keys and values side by side in a page.
    side = dict(v_cache=A + 2 * 64, k_page=4096, v_page=4096, k_slot=256, v_slot=256, k_head=128, v_head=128)
    assert append(**side) != BAD


def test_windows_wider_than_a_c_int(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(sv, "_need_cuda", lambda t, name: None)
    monkeypatch.setattr(sv, "_stream_on", lambda stream, device: 0)
    i32 = torch.int32
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    arrays = (k, k.clone(), torch.zeros(1, 3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32))
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    for window, want in ((0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                         (2 ** 32, 2 ** 31 - 1), (2 ** 32 + 7, 2 ** 31 - 1), (-1, -1), (-2 ** 32, -1)):
        bound = sv.PagedCache(*arrays, q=q, window=window)
        assert sv.lib().spec_paged_attention.argtypes[7] is ctypes.c_int
        assert ctypes.c_int(bound._attend_args[7]).value == want


def test_the_first_truncation_allocates_on_its_own_stream(monkeypatch):
    torch = pytest.importorskip("torch")
    streams = []

    def alloc_on(stream, device):
        streams.append(stream)
        return contextlib.nullcontext()

    monkeypatch.setattr(sv, "_need_cuda", lambda t, name: None)
    monkeypatch.setattr(sv, "_stream_on", lambda stream, device: 77)  # the current one when it is made
    monkeypatch.setattr(sv, "_alloc_on", alloc_on)
    sampler = sv.Sampler(torch.zeros(2, 3, 50), torch.ones(2))
    monkeypatch.setattr(sv, "_stream_on", lambda stream, device: 99)
    sampler._truncate = lambda *args: 0 if args[-1] == 77 else 1
    assert sampler.truncate().shape == (2, 3, 50)
    assert streams == [77]
