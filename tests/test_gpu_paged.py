"""The paged cache: append and attention against double precision.

Bounds: the result's rounding (bf16: 2^-8 of it), the weights' (2^-8 of sum p |v|), and the
scores', whose error e moves every weight by up to 2 e: products of bf16 are exact in single
precision, sums of D of them are off by at most 2 D 2^-24 of the terms' sizes (twice, for
sums that cut instead of rounding).
"""

import math

import pytest

torch = pytest.importorskip("torch")

import round_ref as ref
import speculative_decoding_verification_58_gb300 as sv

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


class Batch:
    """Requests of (new tokens, entries with them), their pages anywhere in the pool."""

    def __init__(self, sizes, Hk=2, G=4, D=128, P=16, seed=1, spare=3, layout="slots", fill=None,
                 sharp=1.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.g, self.sizes, self.Hk, self.H, self.D, self.P = g, sizes, Hk, Hk * G, D, P
        pages = [-(-t // P) for _, t in sizes]
        pool = sum(pages) + spare
        order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
        self.table = torch.full((len(sizes), max(pages) + 2), -1, dtype=torch.int32, device=DEV)
        # What no request uses may hold anything.
        self.table[:, -1] = 2 ** 31 - 1
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        # What the pages hold past a request's entries: NaN unless a value is asked for.
        fill = math.nan if fill is None else fill

        def cache():
            if layout == "heads":  # [pages, heads, slots, width]
                return torch.full((pool, Hk, P, D), fill, dtype=BF, device=DEV).transpose(1, 2)
            return torch.full((pool, P, Hk, D), fill, dtype=BF, device=DEV)

        if layout == "together":  # keys and values of a page side by side
            both = torch.full((pool, 2, P, Hk, D), fill, dtype=BF, device=DEV)
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k, self.v = cache(), cache()
        for b, (_, t) in enumerate(sizes):
            at = torch.arange(t, device=DEV)
            page, slot = self.table[b][at // P].long(), at % P
            self.k[page, slot] = torch.randn((t, Hk, D), generator=g, device=DEV).to(BF)
            self.v[page, slot] = torch.randn((t, Hk, D), generator=g, device=DEV).to(BF)
        starts = [0]
        for n, _ in sizes:
            starts.append(starts[-1] + n)
        self.rows, self.starts = starts[-1], starts
        self.new_start = torch.tensor(starts, dtype=torch.int32, device=DEV)
        self.kv_len = torch.tensor([t for _, t in sizes], dtype=torch.int32, device=DEV)
        self.q = (sharp * torch.randn((max(1, self.rows), self.H, D), generator=g,
                                      device=DEV)).to(BF)

    def arrays(self):
        return self.k, self.v, self.table, self.new_start, self.kv_len

    def check(self, out, lse, causal=True, window=0, scale=None, only=None):
        scale = self.D ** -0.5 if scale is None else scale
        for b, (n, t) in enumerate(self.sizes):
            if n == 0 or (only is not None and b not in only):
                continue
            r = slice(self.starts[b], self.starts[b + 1])
            k = ref.paged_entries(self.k, self.table[b], t)
            v = ref.paged_entries(self.v, self.table[b], t)
            want, want_l, mass, size = ref.attention(self.q[r].double(), k, v, causal, window, scale)
            e = 2 * self.D * 2.0 ** -24 * size
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -16 + 2 * e[..., None]) * mass + 1e-30
            err = (out[r].double() - want).abs()
            assert bool((err <= tol).all()), (b, n, t, float((err / tol).max()),
                                              torch.nonzero(~(err <= tol))[:5].tolist())
            if lse is not None:
                none = want_l == -math.inf
                assert torch.equal(lse[r] == -math.inf, none)
                d = (lse[r].double() - want_l).abs()
                tol = e + 2.0 ** -20 * (1 + want_l.abs())
                assert bool((d <= tol)[~none].all()), (b, n, t, float(d[~none].max()))

    def run(self, causal=True, window=0, scale=None):
        out, lse = sv.spec_paged_attention(self.q, *self.arrays(), causal=causal, window=window,
                                           scale=scale, need_lse=True)
        self.check(out, lse, causal, window, scale)
        return out, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("total", [1, 2, 7, 8, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000])
def test_single_tokens(total, causal, D):
    Batch([(1, total), (1, max(1, total // 2)), (1, total + 3)], D=D).run(causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hk,G,D,P", [(1, 1, 64, 8), (1, 8, 128, 16), (2, 3, 128, 32), (4, 5, 64, 64),
                                      (3, 7, 64, 128), (1, 32, 128, 256), (2, 1, 128, 1024),
                                      (1, 128, 64, 16), (1, 130, 64, 16), (8, 4, 128, 16)])
def test_heads_widths_and_pages(Hk, G, D, P, causal):
    sizes = [(5, 5), (17, 300), (1, 129), (9, 1025), (16, 128)]
    Batch(sizes, Hk=Hk, G=G, D=D, P=P, seed=Hk * 100 + G).run(causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,t", [(2, 2), (31, 40), (32, 500), (33, 33), (63, 64), (64, 64), (65, 700),
                                 (128, 128), (129, 129), (200, 1111), (333, 333), (513, 2000)])
def test_chunks(n, t, causal):
    Batch([(n, t)], Hk=2, G=4).run(causal)
    Batch([(n, t), (1, 50), (n // 2 + 1, t + 77)], Hk=1, G=3, D=64, P=32).run(causal)


@pytest.mark.parametrize("window", [1, 2, 16, 127, 128, 129, 300, 5000])
def test_windows(window):
    Batch([(1, 1000), (17, 600), (40, 40), (130, 900), (1, 3)]).run(True, window)
    Batch([(300, 1300)], D=64, Hk=1, G=2).run(True, window)


def test_rows_that_see_nothing():
    # Fewer entries than new tokens: the first tokens see none.
    for D in (64, 128):
        b = Batch([(9, 4), (3, 0), (150, 20), (2, 300), (1, 0)], D=D)
        out, lse = b.run(True)
        assert bool((out[:5] == 0).all()) and bool((lse[:5] == -math.inf).all())
        assert bool((out[9:12] == 0).all())
        out, lse = b.run(False)
        assert bool((lse[9:12] == -math.inf).all()) and bool((out[9:12] == 0).all())


def test_empty_requests_and_rows_of_nobody():
    b = Batch([(0, 100), (3, 70), (0, 0), (2, 16), (0, 5)])
    rows = b.rows + 6
    q = torch.full((rows, b.H, b.D), math.nan, dtype=BF, device=DEV)
    q[:b.rows] = b.q
    out = torch.full_like(q, 7.0)
    lse = torch.full((rows, b.H), 5.0, device=DEV)
    sv.spec_paged_attention(q, *b.arrays(), out=out, lse=lse)
    b.check(out, lse)
    assert bool((out[b.rows:] == 7.0).all()) and bool((lse[b.rows:] == 5.0).all())
    # Rows before the first request's.
    q[2:2 + b.rows] = b.q
    out.fill_(7.0)
    lse.fill_(5.0)
    sv.spec_paged_attention(q, b.k, b.v, b.table, b.new_start + 2, b.kv_len, out=out, lse=lse)
    b.check(out[2:], lse[2:])
    assert bool((out[:2] == 7.0).all()) and bool((out[2 + b.rows:] == 7.0).all())


@pytest.mark.parametrize("layout", ["heads", "together"])
@pytest.mark.parametrize("P", [8, 64])
def test_cache_layouts(layout, P):
    b = Batch([(17, 400), (1, 90)], P=P, layout=layout)
    b.run(True)
    b.run(False)


def test_rows_of_a_fused_projection():
    b = Batch([(17, 400), (3, 90)])
    out, lse = b.run(True)
    H, Hk, D = b.H, b.Hk, b.D
    qkv = torch.randn((b.rows, H + 2 * Hk, D), device=DEV).to(BF)
    qkv[:, :H] = b.q
    q = qkv[:, :H]
    assert torch.equal(sv.spec_paged_attention(q, *b.arrays()), out)
    k_new, v_new = qkv[:, H:H + Hk], qkv[:, H + Hk:]
    sv.spec_kv_append(k_new, v_new, *b.arrays())
    for i, (n, t) in enumerate(b.sizes):
        r = slice(b.starts[i], b.starts[i + 1])
        assert torch.equal(ref.paged_entries(b.k, b.table[i], t)[t - n:], k_new[r].double())
        assert torch.equal(ref.paged_entries(b.v, b.table[i], t)[t - n:], v_new[r].double())
    b.run(True)


@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf, torch.finfo(BF).min])
def test_what_lies_past_the_entries_is_not_used(fill):
    sizes = [(1, 5), (17, 130), (3, 259), (2, 8), (1, 0)]
    for P in (8, 128):
        for D in (64, 128):
            b = Batch(sizes, P=P, D=D, fill=fill)
            out, lse = b.run(True)
            b.run(False)
            b2 = Batch(sizes, P=P, D=D, fill=0.0)
            assert torch.equal(b2.run(True)[0], out)


@pytest.mark.parametrize("odd", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 3), (True, 40), (True, 200),
                                           (False, 0)])
@pytest.mark.parametrize("D,G,P", [(128, 4, 16), (64, 2, 64), (128, 1, 256)])
def test_values_that_some_rows_do_not_see(D, G, P, causal, window, odd):
    """A value that is not finite is met by its dimension's results of the rows that see it, and
    by nothing else: the other results are those of a 0 in its place."""
    sizes = [(6, 300), (6, 6), (1, 77), (20, 400), (31, 31), (100, 300), (300, 520), (2, 130)]
    b = Batch(sizes, Hk=2, G=G, D=D, P=P, seed=11)
    spots = []  # request, entry, head, dimension
    for i, (n, t) in enumerate(sizes):
        for j, x in enumerate({t - 1, t - n, t - n // 2 - 1, max(0, t - n - 20), t // 3}):
            spots.append((i, x, j % 2, (7 * j + 13 * i) % D))
    v = b.v.clone()

    def put(what):
        b.v.copy_(v)
        for i, x, h, d in spots:
            b.v[b.table[i, x // P].long(), x % P, h, d] = what

    put(0.0)
    want, lse = b.run(causal, window)
    want = want.clone()
    for i, x, h, d in spots:
        n, t = sizes[i]
        for k in range(n):
            at = t - n + k
            if not causal or (x <= at and (window == 0 or x > at - window)):
                want[b.starts[i] + k, h * G:(h + 1) * G, d] += odd
    put(odd)
    out, l2 = sv.spec_paged_attention(b.q, *b.arrays(), causal=causal, window=window, need_lse=True)
    assert torch.equal(lse, l2)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))


@pytest.mark.parametrize("odd", [math.nan, math.inf])
@pytest.mark.parametrize("window", [0, 3, 150])
def test_keys_that_some_rows_do_not_see(window, odd):
    sizes = [(6, 300), (20, 400), (100, 300), (300, 520)]
    b = Batch(sizes, Hk=2, G=4, seed=12)
    want, lse = b.run(True, window)
    k = b.k.clone()
    for i, (n, t) in enumerate(sizes):
        x = t - n // 2 - 1
        b.k[b.table[i, x // b.P].long(), x % b.P] = odd
    out, l2 = sv.spec_paged_attention(b.q, *b.arrays(), causal=True, window=window, need_lse=True)
    for i, (n, t) in enumerate(sizes):
        at = torch.arange(t - n, t, device=DEV)
        x = t - n // 2 - 1
        rows = b.starts[i] + torch.nonzero((at >= x) & ((at - window < x) if window else True))[:, 0]
        if math.isnan(odd):
            assert bool(torch.isnan(out[rows]).all()) and bool(torch.isnan(l2[rows]).all())
        out[rows], l2[rows] = want[rows], lse[rows]
    b.k.copy_(k)
    b.check(out, l2, True, window)


@pytest.mark.parametrize("sharp", [0.01, 8.0, 64.0])
def test_flat_and_sharp_scores(sharp):
    b = Batch([(1, 2000), (17, 700), (150, 150)], sharp=sharp)
    b.run(True)
    b.run(False, scale=0.5)


def test_growing_scores():
    """The largest score comes last, first, or in the middle: the running maximum moves."""
    for direction in (1.0, -1.0):
        b = Batch([(2, 1500), (20, 900)], Hk=1, G=2)
        for i, (_, t) in enumerate(b.sizes):
            at = torch.arange(t, device=DEV)
            page, slot = b.table[i][at // b.P].long(), at % b.P
            grow = direction * (at.float() / t - 0.5)[:, None, None]
            b.k[page, slot] = (0.1 * b.k[page, slot].float() + 4.0 * grow).to(BF)
        b.q.copy_(b.q.float().abs().to(BF))
        b.run(True)
        b.run(False, scale=1.0)


def test_many_requests_of_mixed_lengths():
    g = torch.Generator().manual_seed(3)
    n = torch.randint(0, 20, (200,), generator=g).tolist()
    t = torch.randint(0, 700, (200,), generator=g).tolist()
    b = Batch([(x, max(x, y)) for x, y in zip(n, t)], Hk=2, G=4, D=64, P=32)
    b.run(True)
    b.run(False)


def test_more_requests_than_threads():
    g = torch.Generator().manual_seed(5)
    for B in (385, 1500):
        n = torch.randint(0, 6, (B,), generator=g).tolist()
        t = torch.randint(0, 200, (B,), generator=g).tolist()
        b = Batch([(x, max(x, y)) for x, y in zip(n, t)], Hk=1, G=2, D=64, P=16)
        out, lse = sv.spec_paged_attention(b.q, *b.arrays(), need_lse=True)
        b.check(out, lse, only=set(range(0, B, 7)) | {B - 1})
        again = sv.spec_paged_attention(b.q, *b.arrays())
        assert torch.equal(out, again)


def test_units_of_all_kinds_in_turn():
    """Small and large units next to each other in one CTA: their queries and weights take the
    same shared memory."""
    sizes = []
    for i in range(40):
        sizes += [(1, 3 + i), (100, 140), (20, 30), (1, 1), (40, 41), (70, 200 + i), (2, 600)]
    for D in (64, 128):
        b = Batch(sizes, Hk=2, G=4, D=D, P=64)
        out, lse = sv.spec_paged_attention(b.q, *b.arrays(), need_lse=True)
        b.check(out, lse, only=set(range(0, len(sizes), 5)) | {1, 2, 3, 4})


def test_shared_pages():
    """Requests with a common prefix name the same pages."""
    b = Batch([(3, 200), (5, 210), (1, 140)], P=32)
    for i in (1, 2):
        b.table[i, :4] = b.table[0, :4]
    b.run(True)
    b.run(False)


def test_long_context():
    b = Batch([(1, 100003), (17, 65537)], Hk=2, G=4, P=64)
    b.run(True)
    b.run(True, window=4096)


def test_append_leaves_the_rest():
    for layout in ("slots", "heads", "together"):
        b = Batch([(3, 20), (0, 9), (17, 17), (1, 1000), (40, 65)], Hk=3, G=1, D=64, layout=layout,
                  fill=3.0)
        rows = b.rows + 2
        k_new = torch.randn((rows, b.Hk, b.D), device=DEV).to(BF)
        v_new = torch.randn((rows, b.Hk, b.D), device=DEV).to(BF)
        want_k, want_v = b.k.clone(), b.v.clone()
        for i, (n, t) in enumerate(b.sizes):
            at = torch.arange(t - n, t, device=DEV)
            page, slot = b.table[i][at // b.P].long(), at % b.P
            want_k[page, slot] = k_new[b.starts[i]:b.starts[i + 1]]
            want_v[page, slot] = v_new[b.starts[i]:b.starts[i + 1]]
        k, v = sv.spec_kv_append(k_new, v_new, *b.arrays())
        assert k is b.k and v is b.v
        assert torch.equal(b.k, want_k) and torch.equal(b.v, want_v)


def test_bad_requests():
    sizes = [(3, 20), (2, 40), (17, 300), (1, 50), (4, 30)]

    def fresh():
        b = Batch(sizes, fill=0.5)
        ws = torch.zeros(int(sv.lib().spec_paged_attention_workspace_bytes(
            b.rows, b.H, b.Hk, b.D)), dtype=torch.uint8, device=DEV)
        return b, ws

    b, ws = fresh()
    out, lse = sv.spec_paged_attention(b.q, *b.arrays(), need_lse=True, workspace=ws)
    assert sv.spec_verify_device_status(ws) == sv.SPEC_OK
    good = out.clone()
    for fault in ("len", "negative", "page", "page_low"):
        b, ws = fresh()
        if fault == "len":
            b.kv_len[2] = b.table.shape[1] * b.P + 1
        elif fault == "negative":
            b.kv_len[2] = -1
        elif fault == "page":
            b.table[2, 0] = b.k.shape[0]
        else:
            b.table[2, 18] = -5
        before = b.k.clone(), b.v.clone()
        out, lse = sv.spec_paged_attention(b.q, *b.arrays(), need_lse=True, workspace=ws)
        assert sv.spec_verify_device_status(ws) == sv.SPEC_ERR_BAD_INPUT, fault
        r = slice(b.starts[2], b.starts[3])
        last = b.starts[3] - 1  # sees every page
        assert bool(torch.isnan(out[last]).all()) and bool(torch.isnan(lse[last]).all()), fault
        if fault in ("len", "negative"):
            assert bool(torch.isnan(out[r]).all())
        for i in (0, 1, 3, 4):
            s = slice(b.starts[i], b.starts[i + 1])
            assert torch.equal(out[s], good[s]), (fault, i)
        # The append leaves such a request, or such a token, out.
        new = torch.ones((b.rows, b.Hk, b.D), dtype=BF, device=DEV)
        sv.spec_kv_append(new, new, *b.arrays())
        touched = (b.k != before[0]).any(-1).any(-1)
        pages = b.table[2][(b.table[2] >= 0) & (b.table[2] < b.k.shape[0])].long()
        if fault in ("len", "negative"):
            assert not bool(touched[pages].any())
    # Rows out of range.
    for starts in ([-1, 3, 5, 22, 23, 27], [0, 3, 5, 22, 23, 28], [0, 3, 5, 4, 23, 27]):
        b, ws = fresh()
        b.new_start.copy_(torch.tensor(starts, dtype=torch.int32, device=DEV))
        sv.spec_paged_attention(b.q, *b.arrays(), workspace=ws)
        assert sv.spec_verify_device_status(ws) == sv.SPEC_ERR_BAD_INPUT
        new = torch.ones((b.rows, b.Hk, b.D), dtype=BF, device=DEV)
        sv.spec_kv_append(new, new, *b.arrays())
    torch.cuda.synchronize()


def test_past_32_bit_offsets():
    """A cache of more than 2^32 entries, the request's pages at its end."""
    Hk, D, P = 8, 128, 64
    pool = (1 << 32) // (Hk * D * P) + 50
    k = torch.zeros((pool, P, Hk, D), dtype=BF, device=DEV)
    v = torch.zeros((pool, P, Hk, D), dtype=BF, device=DEV)
    b = Batch([(17, 900)], Hk=Hk, D=D, P=P)
    far = torch.arange(pool - 16, pool, dtype=torch.int32, device=DEV)
    used = b.table[0, :15].long()
    k[far[:15].long()], v[far[:15].long()] = b.k[used], b.v[used]
    table = torch.full((1, 16), -1, dtype=torch.int32, device=DEV)
    table[0, :15] = far[:15]
    new = torch.randn((b.rows, Hk, D), device=DEV).to(BF)
    b.k, b.v, b.table = k, v, table
    sv.spec_kv_append(new, new, *b.arrays())
    at = torch.arange(900 - 17, 900, device=DEV)
    assert torch.equal(k[table[0][at // P].long(), at % P], new)
    b.run(True)


def test_graph_streams_and_bound_form():
    b = Batch([(5, 300), (17, 900), (1, 64)])
    new = torch.randn((b.rows, b.Hk, b.D), device=DEV).to(BF)
    bound = sv.PagedCache(*b.arrays(), k_new=new, v_new=new, q=b.q, need_lse=True)
    bound.append()
    out, lse = (t.clone() for t in bound.attend())
    b.check(out, lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = sv.spec_paged_attention(b.q, *b.arrays(), stream=side)
    side.synchronize()
    assert torch.equal(out, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # (an object is bound to the stream it is made on)
        bound = sv.PagedCache(*b.arrays(), k_new=new, v_new=new, q=b.q, need_lse=True)
        bound.append()
        o2, l2 = bound.attend()
    for seed in (1, 2):
        new.copy_(torch.randn(new.shape, generator=b.g, device=DEV).to(BF))
        b.q.copy_(torch.randn(b.q.shape, generator=b.g, device=DEV).to(BF))
        b.kv_len.sub_(seed)  # other lengths than the graph was captured with
        b.sizes = [(n, t - seed) for n, t in b.sizes]
        graph.replay()
        torch.cuda.synchronize()
        b.check(o2, l2)


def test_same_bits_on_every_call():
    b = Batch([(17, 5000), (1, 9000), (200, 3000)], Hk=2, G=4)
    one = sv.spec_paged_attention(b.q, *b.arrays(), need_lse=True)
    for _ in range(3):
        two = sv.spec_paged_attention(b.q, *b.arrays(), need_lse=True)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
