"""A round as a serving loop makes it: draft tokens drawn under the requests' settings, the new
tokens' keys and values appended, attention over the cache, both sides' logits truncated, verified
and the next block selected; eager, on two streams at once, and as a replayed graph."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
import round_ref as ref
import speculative_decoding_verification_58_gb300 as sv

pytestmark = pytest.mark.gpu

DEV, BF = "cuda", torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


class Round:
    """A toy target and drafter: random projections around the library's calls."""

    def __init__(self, B, k, V, seed, Hk=2, G=4, D=64, P=16, context=200, stream=None):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.B, self.k, self.V, self.Hk, self.H, self.D, self.P = B, k, V, Hk, Hk * G, D, P
        rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        n = k + 1
        pages = -(-(context + 4 * n) // P)
        self.k_cache = rnd(B * pages + 3, P, Hk, D).to(BF)
        self.v_cache = rnd(B * pages + 3, P, Hk, D).to(BF)
        order = torch.randperm(B * pages + 3, generator=g, device=DEV)[:B * pages]
        self.table = order.to(torch.int32).view(B, pages).contiguous()
        old = torch.randint(1, context, (B,), generator=g, device=DEV)
        self.new_start = (torch.arange(B + 1, device=DEV) * n).to(torch.int32)
        self.kv_len = (old + n).to(torch.int32)
        self.qkv = rnd(B * n, self.H + 2 * Hk, D).to(BF)
        self.head = (rnd(self.H * D, V) / math.sqrt(self.H * D) * 4.0).to(BF)
        self.noise = 0.5 * rnd(B, k, V)
        self.temperature = torch.tensor([0.7, 1.0, 0.0, 1.2] * B, device=DEV)[:B].contiguous()
        self.top_k = torch.tensor([0, 40, 0, 7] * B, dtype=torch.int32, device=DEV)[:B].contiguous()
        self.top_p = torch.tensor([0.9, 1.0, 1.0, 0.95] * B, device=DEV)[:B].contiguous()
        self.min_p = torch.tensor([0.0, 0.02, 0.0, 0.0] * B, device=DEV)[:B].contiguous()
        self.u_draft = torch.rand((B, k), generator=g, device=DEV)
        self.u = torch.rand((B, k + 1), generator=g, device=DEV)
        self.lengths = torch.randint(1, k + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        self.stream = stream

    def run(self):
        kw = dict(top_k=self.top_k, top_p=self.top_p, min_p=self.min_p, stream=self.stream)
        H, Hk = self.H, self.Hk
        paged = (self.k_cache, self.v_cache, self.table, self.new_start, self.kv_len)
        sv.spec_kv_append(self.qkv[:, H:H + Hk], self.qkv[:, H + Hk:], *paged, stream=self.stream)
        out = sv.spec_paged_attention(self.qkv[:, :H], *paged, stream=self.stream)
        target = (out.flatten(1) @ self.head).view(self.B, self.k + 1, self.V)
        draft = (target[:, :self.k].float() + self.noise).to(BF)
        tokens, q = sv.spec_sample(draft, self.temperature, self.u_draft, kept=torch.empty_like(draft),
                                   **kw)
        p = sv.spec_truncate(target, self.temperature, kept=target.clone(), **kw)
        got, n = sv.spec_verify(p, q, tokens, self.lengths, self.u, self.temperature,
                                stream=self.stream)
        return dict(out=out, target=target, draft=draft, tokens=tokens, q=q, p=p, got=got, n=n)

    def check(self, r):
        B, k = self.B, self.k
        n = k + 1
        for b in range(B):
            t = int(self.kv_len[b])
            kk = ref.paged_entries(self.k_cache, self.table[b], t)
            vv = ref.paged_entries(self.v_cache, self.table[b], t)
            rows = slice(b * n, (b + 1) * n)
            assert torch.equal(kk[t - n:], self.qkv[rows, self.H:self.H + self.Hk].double())
            assert torch.equal(vv[t - n:], self.qkv[rows, self.H + self.Hk:].double())
            want, _, mass, size = ref.attention(self.qkv[rows, :self.H].double(), kk, vv, True, 0,
                                                self.D ** -0.5)
            e = 2 * self.D * 2.0 ** -24 * size
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -16 + 2 * e[..., None]) * mass + 1e-30
            assert bool(((r["out"][rows].double() - want).abs() <= tol).all())
            a = (float(self.temperature[b]), int(self.top_k[b]), float(self.top_p[b]),
                 float(self.min_p[b]))
            for i in range(n):
                keep, w, near = ref.truncate(r["target"][b, i], *a)
                if not near:
                    assert torch.equal(r["p"][b, i] > -math.inf, keep)
                if i < k:
                    keep, w, near = ref.truncate(r["draft"][b, i], *a)
                    tok, near_u = ref.draw(w, float(self.u_draft[b, i]))
                    if not near and not near_u:
                        assert int(r["tokens"][b, i]) == tok
                    # A drawn token has mass in the distribution it came from.
                    assert float(r["q"][b, i, int(r["tokens"][b, i])]) > -math.inf
        # Verification of the truncated rows, against the oracle on the same rows.
        bits = lambda x: x.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
        o = oracle.verify(bits(r["p"]), bits(r["q"]), r["tokens"].cpu().numpy(),
                          self.lengths.cpu().numpy(), self.u.cpu().numpy(),
                          self.temperature.cpu().numpy())
        got, num = r["got"].cpu().numpy(), r["n"].cpu().numpy()
        near = o.margin < 1e-6
        same = (num == o.num_accepted) & np.all(got == o.out_tokens, axis=1)
        assert np.all(same | near), (num, o.num_accepted)
        assert np.all(num >= 0)
        # What is emitted was kept.
        for b in range(B):
            last = int(got[b, num[b]])
            assert float(r["p"][b, num[b], last]) > -math.inf


@pytest.mark.parametrize("B,k,V", [(1, 4, 500), (6, 16, 3001), (9, 3, 32000)])
def test_rounds(B, k, V):
    r = Round(B, k, V, seed=B)
    res = r.run()
    torch.cuda.synchronize()
    r.check(res)
    # The next round: the accepted tokens and the emitted one stay, the others' entries are
    # written over.
    r.kv_len.add_(res["n"] + 1)
    r.qkv.copy_(torch.randn(r.qkv.shape, device=DEV).to(BF))
    res = r.run()
    torch.cuda.synchronize()
    r.check(res)


def test_two_rounds_on_two_streams():
    a, b = Round(5, 8, 4000, seed=1), Round(7, 5, 9000, seed=2, D=128)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    results = []
    for r, s in zip((a, b), streams):
        s.wait_stream(torch.cuda.current_stream())
        r.stream = None
        with torch.cuda.stream(s):
            results.append([r.run() for _ in range(3)][-1])
    torch.cuda.synchronize()
    a.check(results[0])
    b.check(results[1])


def test_a_round_as_a_graph():
    r = Round(6, 7, 5000, seed=3)
    r.run()  # (sets the kernels up)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = r.run()
    for seed in (5, 6):
        g = torch.Generator(device=DEV).manual_seed(seed)
        r.qkv.copy_(torch.randn(r.qkv.shape, generator=g, device=DEV).to(BF))
        r.u.copy_(torch.rand(r.u.shape, generator=g, device=DEV))
        r.top_k.copy_(torch.randint(0, 60, (r.B,), generator=g, device=DEV).to(torch.int32))
        r.lengths.copy_(torch.randint(1, r.k + 1, (r.B,), generator=g, device=DEV).to(torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        r.check(res)


def test_truncated_sampling_is_lossless():
    """Over many draws, what a round emits first is distributed as the truncated target."""
    B, V, k = 20000, 12, 1
    g = torch.Generator(device=DEV).manual_seed(4)
    zt = torch.randn((1, k + 1, V), generator=g, device=DEV).expand(B, k + 1, V).contiguous()
    zd = (zt[:, :k] + 0.8 * torch.randn((1, k, V), generator=g, device=DEV)).contiguous()
    T = torch.full((B,), 0.9, device=DEV)
    kw = dict(top_k=torch.full((B,), 7, dtype=torch.int32, device=DEV),
              top_p=torch.full((B,), 0.9, device=DEV))
    tokens, q = sv.spec_sample(zd, T, torch.rand((B, k), generator=g, device=DEV),
                               kept=torch.empty_like(zd), **kw)
    p = sv.spec_truncate(zt, T, **kw)
    out, n = sv.spec_verify(p, q, tokens, torch.ones(B, dtype=torch.int32, device=DEV),
                            torch.rand((B, k + 1), generator=g, device=DEV), T)
    keep, w, near = ref.truncate(zt[0, 0], 0.9, 7, 0.9)
    assert not near
    want = (w / w.sum()).cpu()
    freq = torch.bincount(out[:, 0].long(), minlength=V).double().cpu() / B
    assert bool((freq[~keep.cpu()] == 0).all())
    # Five standard deviations of each frequency.
    assert bool(((freq - want).abs() <= 5 * (want * (1 - want) / B).sqrt() + 1e-9).all())
