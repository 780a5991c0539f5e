"""The training calls as a loop uses them, after a verification round (needs a GB300).

A draft head reads hidden states; its logits are verified against the target's; the
statistics give the labels; the mixture loss's gradient goes back through the
head by an ordinary product, the hard-label loss through spec_linear_ce_grad;
all gradients are clipped together.  Each result is compared with double precision
on the inputs that the call before it produced (tolerances as derived in the single
operators' tests).
"""

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_58_gb300 as sv
import train_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.lib()


def make(B, k, V, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn((V, D), generator=g, device="cuda") * (2.0 / D ** 0.5)).to(torch.bfloat16)
    h = torch.randn((B, k, D), generator=g, device="cuda").to(torch.bfloat16)
    draft = (h.reshape(-1, D) @ w.t()).reshape(B, k, V)  # bf16 logits
    target = torch.empty((B, k + 1, V), dtype=torch.bfloat16, device="cuda")
    target[:, :k] = draft + 0.5 * torch.randn((B, k, V), generator=g, device="cuda")
    target[:, k] = torch.randn((B, V), generator=g, device="cuda")
    L = torch.randint(1, k + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    tok = draft.float().argmax(2).to(torch.int32)
    u = torch.rand((B, k + 1), generator=g, device="cuda")
    T = torch.ones(B, device="cuda")
    return w, h, draft, target, L, tok, u, T


def step(w, h, draft, target, L, tok, u, T, bufs):
    """One round and one training step into fixed buffers; what a loop runs."""
    B, k, D = h.shape
    sv.spec_verify(target, draft, tok, L, u, T, workspace=bufs["ws"], out_tokens=bufs["out"],
                   num_accepted=bufs["n"])
    sv.spec_opd_stats(target, draft, L, out=bufs["stats"])
    # Labels: the target's argmax, -1 past a request's length.
    bufs["labels"].copy_(bufs["stats"].x_star.reshape(-1))
    sv.spec_opd_grad(target, draft, L, bufs["g_loss"], d_draft=bufs["dz"])
    bufs["ce"].loss()
    bufs["ce"].grad()
    torch.mm(bufs["dz"].reshape(B * k, -1), w, out=bufs["dh2"])
    bufs["clip"]()


def buffers(w, h, draft, target, L):
    B, k, D = h.shape
    V = w.shape[0]
    dev = "cuda"
    b = {"ws": sv.alloc_workspace(B, k, V), "out": torch.empty((B, k + 1), dtype=torch.int32, device=dev),
         "n": torch.empty(B, dtype=torch.int32, device=dev),
         "labels": torch.empty(B * k, dtype=torch.int32, device=dev),
         "g_loss": torch.full((B,), 1.0 / B, device=dev), "dz": torch.empty_like(draft),
         "dh2": torch.empty((B * k, D), dtype=torch.bfloat16, device=dev)}
    f = dict(dtype=torch.float32, device=dev)
    b["stats"] = sv.OpdStats(torch.empty((B, k), dtype=torch.int32, device=dev), torch.empty((B, k), **f),
                             torch.empty((B, k), **f), torch.empty((B, k), **f), torch.empty(B, **f))
    # Weights that fall with the position in the block.
    gn = torch.exp(-torch.arange(k, device=dev) / 7.0).repeat(B) / (B * k)
    b["gn"] = gn
    b["ce"] = sv.LinearCe(h.reshape(B * k, D), w, b["labels"], gn)
    b["out_g"] = [torch.empty_like(t) for t in (b["ce"].d_hidden, b["ce"].d_weight, b["dh2"])]
    b["clip"] = sv.GradClipper([b["ce"].d_hidden, b["ce"].d_weight, b["dh2"]], 0.01, out=b["out_g"])
    return b


def check(w, h, draft, target, L, b):
    B, k, D = h.shape
    hh = h.reshape(B * k, D)
    x = b["stats"].x_star
    for i in range(B):
        Li = int(L[i])
        assert torch.equal(x[i, :Li].long(), target[i, :Li].float().argmax(1))
        assert torch.all(x[i, Li:] == -1)
    assert torch.all(b["n"] >= 0)
    y = b["labels"]
    rn, rl = ref.ce(hh, w, y)
    assert torch.allclose(b["ce"].nll.double(), rn, rtol=1e-4, atol=1e-4)
    rh, rw, dz, mass = ref.ce_grad(hh, w, y, b["gn"])
    for got, want, mag in ((b["ce"].d_hidden, rh, dz.abs() @ w.double().abs()),
                           (b["ce"].d_weight, rw, dz.abs().t() @ hh.double().abs())):
        assert torch.all((got.double() - want).abs() <= 2.0 ** -8 * 1.1 * mag + 2.0 ** -8 * want.abs()
                         + 1e-3 * mag.mean())
    want, scale, logq, _ = ref.opd_grad(target, draft, L, b["g_loss"], 0.01, 0.8)
    flip, _, _, at_clip = ref.opd_grad(target, draft, L, b["g_loss"], 0.01, 0.8, 2e-4)
    tol = scale * (2.0 ** -15 + logq.abs() * 2.0 ** -21) + 2.0 ** -8 * want.abs() + 1e-37
    ok = ((b["dz"].double() - want).abs() <= tol).all(2)
    ok |= ((b["dz"].double() - flip).abs() <= tol + 2.0 ** -8 * flip.abs()).all(2) & at_clip
    assert torch.all(ok)
    grads = [b["ce"].d_hidden, b["ce"].d_weight, b["dh2"]]
    norm = ref.norm(grads)
    assert abs(float(b["clip"].norm) - norm) <= 2.0 ** -18 * norm
    f = min(1.0, 0.01 / norm)
    for a, o in zip(grads, b["out_g"]):
        t = a.double() * f
        assert torch.all((o.double() - t).abs() <= (2.0 ** -8 + 2.0 ** -17) * t.abs() + 1e-38)


@pytest.mark.parametrize("B,k,V,D", [(3, 4, 1000, 64), (9, 16, 5003, 136), (16, 7, 32000, 256)])
def test_round_and_step(B, k, V, D):
    args = make(B, k, V, D, seed=B + V)
    b = buffers(*args[:5])
    step(*args, b)
    check(*args[:5], b)


def test_step_as_a_graph_replayed_on_new_data():
    B, k, V, D = 6, 8, 3001, 72
    args = make(B, k, V, D, seed=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = buffers(*args[:5])  # the bound calls take this stream
        step(*args, b)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step(*args, b)
    for seed in (2, 3):
        for dst, src in zip(args, make(B, k, V, D, seed=seed)):
            dst.copy_(src)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(*args[:5], b)


def test_two_loops_on_two_streams():
    # Two independent steps enqueued without waiting for one another give what each
    # gives alone.
    runs = []
    for seed in (11, 12):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            args = make(5, 8, 9001, 200, seed=seed)
            b = buffers(*args[:5])
        runs.append((s, args, b))
    torch.cuda.synchronize()
    for _ in range(4):
        for s, args, b in runs:
            with torch.cuda.stream(s):
                step(*args, b)
    torch.cuda.synchronize()
    for s, args, b in runs:
        check(*args[:5], b)


@pytest.mark.parametrize("handle", [False, True])
def test_calls_given_a_stream_keep_their_memory(handle):
    """What a call allocates for a stream of its own is not handed out while that stream uses it.

    The stream is held up, the calls are enqueued behind that, and their workspaces'
    sizes are allocated and filled from the current stream meanwhile.
    """
    N, V, D = 64, 1024, 128
    w, h, draft, target, L, tok, u, T = make(8, 8, V, D, 3)
    h = h.reshape(N, D)
    y = torch.arange(N, device="cuda", dtype=torch.int32) * 7 % V
    g = torch.full((N,), 1.0 / N, device="cuda")
    gl = torch.full((8,), 0.125, device="cuda")

    def run(stream):
        nll, lse = sv.spec_linear_ce(h, w, y, stream=stream)
        dh, dw = sv.spec_linear_ce_grad(h, w, y, nll, lse, g, stream=stream)
        dz = sv.spec_opd_grad(target, draft, L, gl, stream=stream)
        return nll, lse, dh, dw, dz, sv.spec_grad_norm([h, w], stream=stream)

    want = run(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)  # some 50 ms
    got = run(s.cuda_stream if handle else s)
    sizes = [sv.lib().spec_linear_ce_workspace_bytes(N, V, D),
             sv.lib().spec_linear_ce_grad_workspace_bytes(N, V, D),
             sv.lib().spec_grad_norm_workspace_bytes(2)]
    others = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes * 3]
    s.synchronize()
    torch.cuda.synchronize()
    assert all(bool((t == 255).all()) for t in others)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_range_checking_build():
    """The training calls through libspecverify_debug.so: no index leaves its buffer."""
    code = """
import torch, sys
sys.path.insert(0, {tests!r}); sys.path.insert(0, {root!r})
import speculative_decoding_verification_58_gb300 as sv
import test_gpu_training_run as t
assert sv.spec_debug_build()
sv.spec_debug_checks(reset=True)
for shape in ((3, 4, 1000, 64), (5, 16, 5003, 136), (40, 8, 300, 72)):
    args = t.make(*shape, seed=4)
    b = t.buffers(*args[:5])
    t.step(*args, b)
    t.check(*args[:5], b)
torch.cuda.synchronize()
print("range checks failed:", sv.spec_debug_checks()[0])
""".format(tests=os.path.dirname(os.path.abspath(__file__)),
           root=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, SPEC_VERIFY_DEBUG="1"),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-3000:]
    assert "range checks failed: 0" in r.stdout, r.stdout[-2000:]
