"""Training calls that read what the call right before them wrote (needs a GB300).

The kernels start ahead of their predecessor's end, and two of them read inputs before their own
wait for it.  Each call here takes the buffers of the call before it as they are, with
no copy in between, new contents in every turn and no wait of the host: every result has
to be the one of the same call made alone, to the bit.
"""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


class Loop:
    """Statistics and mixture gradient of a batch; its labels and its gradient as the labels and
    hidden states of a head; that head's loss and gradients; their norm and clip."""

    def __init__(self, B, k, V, rows, seeds):
        self.B, self.k, self.V = B, k, V
        g = torch.Generator(device="cuda").manual_seed(B * k + V)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.data = []
        for _ in range(seeds):
            t = (2 * rnd(B, k + 1, V)).to(torch.bfloat16)
            d = (t[:, :k].float() + rnd(B, k, V)).to(torch.bfloat16)
            # Argmaxima among a few entries: labels that many tokens share.
            top = torch.randint(0, 3, (B, k + 1, 1), generator=g, device="cuda") * 2
            t.scatter_(2, top, 20.0)
            self.data.append((t, d, 0.5 + torch.rand(B, generator=g, device="cuda")))
        self.L = torch.randint(1, k + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        f = dict(dtype=torch.float32, device="cuda")
        self.stats = sv.OpdStats(torch.empty((B, k), dtype=torch.int32, device="cuda"),
                                 torch.empty((B, k), **f), torch.empty((B, k), **f),
                                 torch.empty((B, k), **f), torch.empty(B, **f))
        self.t, self.d, self.gl = (torch.empty_like(x) for x in self.data[0])
        self.dz = torch.empty_like(self.d)
        self.w = (rnd(rows, V) * 4).to(torch.bfloat16)
        N = B * k
        self.head = sv.LinearCe(self.dz.reshape(N, V), self.w, self.stats.x_star.reshape(N),
                                torch.full((N,), 1.0 / N, device="cuda"))
        grads = [self.head.d_hidden, self.head.d_weight]
        self.out = [torch.empty_like(x) for x in grads]
        self.clip = sv.GradClipper(grads, 0.01, out=self.out)

    def turn(self, i, wait=lambda: None):
        t, d, gl = self.data[i]
        for dst, src in ((self.t, t), (self.d, d), (self.gl, gl)):
            dst.copy_(src)
        wait()
        sv.spec_opd_stats(self.t, self.d, self.L, out=self.stats)
        wait()
        sv.spec_opd_grad(self.t, self.d, self.L, self.gl, d_draft=self.dz)
        wait()
        self.head.loss()
        wait()
        self.head.grad()
        wait()
        self.clip()
        wait()

    def results(self):
        s = self.stats
        return [x.clone() for x in (s.x_star, s.loss, self.dz, self.head.nll, self.head.lse,
                                    self.head.d_hidden, self.head.d_weight, self.clip.norm, *self.out)]


SHAPES = [
    (1, 3, 1000, 500),     # a few tokens
    (8, 8, 264, 1024),     # small kernels, all of them beside one another
    (20, 16, 2048, 3000),  # slices of dH
    (40, 16, 136, 151936), # several pieces
]


@pytest.mark.parametrize("B,k,V,rows", SHAPES)
def test_without_waits(B, k, V, rows):
    loop = Loop(B, k, V, rows, 3)
    want = []
    for i in range(3):
        loop.turn(i, torch.cuda.synchronize)
        want.append(loop.results())
    assert not torch.equal(want[0][3], want[1][3])
    assert torch.all(torch.isfinite(want[0][6].float()))
    got = []
    for n in range(30):
        loop.turn(n % 3)
        if n % 4 == 3 or n < 3:
            got.append((n % 3, loop.results()))
    torch.cuda.synchronize()
    for i, r in got:
        for a, b in zip(r, want[i]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("B,k,V,rows", SHAPES)
def test_as_a_graph(B, k, V, rows):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        loop = Loop(B, k, V, rows, 2)
        want = []
        for i in range(2):
            loop.turn(i, torch.cuda.synchronize)
            want.append(loop.results())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for i in (0, 1, 0, 1):
                loop.turn(i)
        for _ in range(5):
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(loop.results(), want[1]):
            assert torch.equal(a, b)


def test_two_loops_beside_one_another():
    runs = []
    for shape in (SHAPES[1], SHAPES[2]):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            loop = Loop(*shape, 2)
            want = []
            for i in range(2):
                loop.turn(i, torch.cuda.synchronize)
                want.append(loop.results())
        runs.append((s, loop, want, []))
    for n in range(20):
        for s, loop, want, got in runs:
            with torch.cuda.stream(s):
                loop.turn(n % 2)
                got.append(loop.results())
    torch.cuda.synchronize()
    for s, loop, want, got in runs:
        for n, r in enumerate(got):
            for a, b in zip(r, want[n % 2]):
                assert torch.equal(a, b)
