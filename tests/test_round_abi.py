"""Sampling, truncation and the paged cache without a GPU: argument checks that return before
any CUDA call, and what the binding refuses."""

import ctypes

import pytest

import speculative_decoding_verification_58_gb300 as sv

A = 1 << 24  # addresses that are never read
BAD, UNS, WSP = sv.SPEC_ERR_INVALID_ARG, sv.SPEC_ERR_UNSUPPORTED, sv.SPEC_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    sv.build()
    return sv.lib()


def test_sample_host_checks(lib):
    def f(z=A, dt=0, rows=4, V=100, group=2, T=2 * A, k=3 * A, p=4 * A, m=5 * A, u=6 * A, tok=7 * A,
          kept=None):
        return lib.spec_sample(z, dt, rows, V, group, T, k, p, m, u, tok, kept, None)

    for kw in (dict(rows=0), dict(V=0), dict(group=0), dict(dt=2), dict(dt=-1), dict(z=None), dict(T=None),
               dict(u=None), dict(tok=None), dict(z=A + 2), dict(dt=1, z=A + 1), dict(T=2 * A + 1),
               dict(k=3 * A + 2), dict(p=4 * A + 2), dict(m=5 * A + 2), dict(u=6 * A + 2),
               dict(tok=7 * A + 2), dict(tok=A), dict(tok=6 * A + 4), dict(tok=2 * A + 4),
               dict(tok=5 * A), dict(kept=A + 4), dict(kept=7 * A), dict(kept=2 * A - 8),
               dict(kept=8 * A + 2), dict(kept=6 * A)):
        assert f(**kw) == BAD, kw
    assert f(V=(1 << 21) + 1) == UNS and f(rows=(1 << 24) + 1) == UNS


def test_truncate_host_checks(lib):
    def f(z=A, dt=1, rows=4, V=100, group=1, T=2 * A, k=None, p=None, m=None, kept=3 * A):
        return lib.spec_truncate(z, dt, rows, V, group, T, k, p, m, kept, None)

    for kw in (dict(kept=None), dict(kept=A + 2), dict(kept=A - 2), dict(T=None), dict(kept=2 * A),
               dict(kept=3 * A + 1), dict(p=3 * A + 4), dict(rows=-1)):
        assert f(**kw) == BAD, kw
    assert f(V=1 << 22) == UNS


def cache(**kw):
    c = dict(k_cache=A, v_cache=2 * A, k_page=16 * 2 * 64, k_slot=2 * 64, k_head=64, v_page=16 * 2 * 64,
             v_slot=2 * 64, v_head=64, num_pages=10, page_size=16, kv_heads=2, width=64,
             page_table=3 * A, max_pages=4, new_start=4 * A, kv_len=5 * A, B=3)
    c.update(kw)
    return sv._PagedCache(*(c[n] for n, _ in sv._PagedCache._fields_))


CACHE_BAD = (dict(k_cache=None), dict(v_cache=None), dict(page_table=None), dict(new_start=None),
             dict(kv_len=None), dict(B=0), dict(num_pages=0), dict(page_size=0), dict(kv_heads=0),
             dict(width=0), dict(max_pages=0), dict(k_cache=A + 8), dict(v_cache=2 * A + 2),
             dict(k_page=56), dict(k_slot=132), dict(v_head=32), dict(v_slot=0), dict(v_page=-64),
             dict(k_page=1 << 39), dict(kv_len=5 * A + 2), dict(page_table=3 * A + 1))
CACHE_UNS = (dict(page_size=4), dict(page_size=24), dict(page_size=2048), dict(width=96),
             dict(width=256), dict(kv_heads=2048), dict(max_pages=1 << 28), dict(B=(1 << 18) + 1))


def test_append_host_checks(lib):
    def f(c=None, dt=1, k=6 * A, v=7 * A, rows=5, ks=128, vs=128, **kw):
        c = cache(**kw) if c is None else c
        return lib.spec_kv_append(ctypes.byref(c), dt, k, v, rows, ks, vs, None)

    assert lib.spec_kv_append(None, 1, 6 * A, 7 * A, 5, 128, 128, None) == BAD
    for kw in CACHE_BAD + (dict(dt=5), dict(k=None), dict(v=None), dict(k=6 * A + 2), dict(rows=0),
                           dict(ks=120), dict(vs=132), dict(ks=-128), dict(k=A + 64), dict(v=2 * A),
                           dict(k=2 * A + 256), dict(page_table=A + 64), dict(kv_len=2 * A + 4)):
        assert f(**kw) == BAD, kw
    for kw in CACHE_UNS + (dict(dt=0), dict(rows=(1 << 24) + 1)):
        assert f(**kw) == UNS, kw


def test_attention_host_checks(lib):
    ws = lib.spec_paged_attention_workspace_bytes
    assert ws(1, 1, 1, 64) > 0 and ws(2048, 32, 8, 128) % 256 == 0
    assert ws(0, 1, 1, 64) == ws(1, 3, 2, 64) == ws(1, 1, 1, 96) == ws(1, 2048, 1, 64) == 0
    assert ws((1 << 24) + 1, 1, 1, 64) == ws(1, 0, 1, 64) == ws(1, 1, 0, 64) == 0

    def f(dt=1, q=6 * A, rows=5, H=4, qs=256, causal=1, window=0, scale=0.1, out=7 * A, lse=8 * A,
          w=9 * A, n=1 << 40, **kw):
        c = cache(**kw)
        return lib.spec_paged_attention(ctypes.byref(c), dt, q, rows, H, qs, causal, window, scale, out,
                                        lse, w, n, None)

    for kw in CACHE_BAD + (dict(dt=3), dict(q=None), dict(out=None), dict(rows=0), dict(H=0), dict(H=3),
                           dict(qs=200), dict(qs=260), dict(causal=2), dict(causal=-1), dict(window=-1),
                           dict(causal=0, window=5), dict(scale=0.0), dict(scale=-1.0),
                           dict(scale=float("nan")), dict(scale=float("inf")), dict(q=6 * A + 8),
                           dict(out=7 * A + 4), dict(lse=8 * A + 2), dict(out=6 * A + 16), dict(out=A),
                           dict(out=2 * A + 32), dict(lse=7 * A), dict(lse=5 * A + 4), dict(out=3 * A),
                           dict(lse=6 * A)):
        assert f(**kw) == BAD, kw
    for kw in CACHE_UNS + (dict(dt=0), dict(H=2048, qs=2048 * 64)):
        assert f(**kw) == UNS, kw
    for kw in (dict(w=None), dict(w=9 * A + 16), dict(n=16)):
        assert f(**kw) == WSP, kw


def test_binding_refusals(monkeypatch):
    torch = pytest.importorskip("torch")
    z, T, u = torch.zeros(2, 3, 50), torch.ones(2), torch.zeros(2, 3)
    with pytest.raises(ValueError):
        sv.spec_sample(z, T, u)  # host tensors
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros(4, 16, 2, 64, dtype=bf)
    table, start, ln = torch.zeros(1, 3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32)
    q = torch.zeros(3, 4, 64, dtype=bf)
    with pytest.raises(ValueError):
        sv.spec_paged_attention(q, k, k.clone(), table, start, ln)
    monkeypatch.setattr(sv, "_need_cuda", lambda t, name: None)
    monkeypatch.setattr(sv, "_stream_on", lambda stream, device: 0)
    with pytest.raises(ValueError, match="uniforms"):
        sv.spec_sample(z, T, None)
    for bad in (dict(logits=z[0, 0]), dict(temperature=torch.ones(3)), dict(top_k=torch.ones(2)),
                dict(top_p=torch.ones(2, dtype=torch.float64)), dict(min_p=torch.ones(6)),
                dict(uniforms=torch.zeros(2)), dict(kept=torch.zeros(2, 3, 49)),
                dict(tokens=torch.zeros(2, 3)), dict(logits=z.half()),
                dict(logits=torch.zeros(2, 50, 3).transpose(1, 2))):
        kw = dict(logits=z, temperature=T, uniforms=u)
        kw.update(bad)
        with pytest.raises((ValueError, TypeError)):
            sv.Sampler(kw.pop("logits"), kw.pop("temperature"), kw.pop("uniforms"), **kw)
    with pytest.raises(ValueError, match="uniforms"):
        sv.Sampler(z, T).sample()
    new = torch.zeros(3, 2, 64, dtype=bf)
    good = (k, k.clone(), table, start, ln)
    for i, bad in ((0, k[0]), (1, k.clone()[:, :8]), (1, k.float()), (2, table[0]), (2, table.long()),
                   (3, start[:1]), (4, ln.long()), (0, k.transpose(2, 3))):
        args = list(good)
        args[i] = bad
        with pytest.raises((ValueError, TypeError)):
            sv.PagedCache(*args, q=q)
    for kw in (dict(k_new=new), dict(k_new=new, v_new=new[:2]), dict(k_new=new.float(), v_new=new),
               dict(q=q[..., :32]), dict(q=q.transpose(0, 1)), dict(q=q, out=q[:2]),
               dict(q=q, lse=torch.zeros(3, 5)), dict(q=q.permute(0, 2, 1))):
        with pytest.raises((ValueError, TypeError)):
            sv.PagedCache(*good, **kw)
    with pytest.raises(ValueError, match="k_new"):
        sv.PagedCache(*good).append()
    with pytest.raises(ValueError, match="q"):
        sv.PagedCache(*good).attend()
    with pytest.raises(ValueError):
        sv.spec_kv_append(None, None, *good)
    with pytest.raises(ValueError):
        sv.spec_paged_attention(None, *good)
