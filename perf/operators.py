"""The drafter-training operators, as cases that can be timed and compared.

Each case is one call of a training loop that distils a drafter on the batch
that verification has just read:

``ce_eval``   token losses of a linear vocabulary head (``spec_linear_ce``):
              nll_i = logsumexp_v(h_i . w_v) - h_i . w_{y_i}
``ce_train``  the same and the gradients of sum_i g_i nll_i with respect to the
              hidden states and the head's weight (``spec_linear_ce_grad``)
``opd_grad``  gradient of the mixture distillation loss with respect to the
              draft logits (``spec_opd_grad``)
``clip``      global norm of many gradient tensors, and the tensors scaled to a
              largest norm (``spec_clip_grad_norm``)

``run`` computes them in elementary torch operations, or through the
library's entry points where ``own`` is true.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DELTA, ALPHA = 0.01, 0.8  # entry-wise clip and mixture weight of the distillation loss
BLOCK = 16                # draft positions per request


def listed():
    return [
        # Loss of one token under a full vocabulary: the latency of a single evaluation.
        {"name": "ce_eval_one_token", "op": "ce_eval", "N": 1, "V": 151936, "D": 1024},
        # Held-out loss of 128 requests of 16 positions.
        {"name": "ce_eval_128_requests", "op": "ce_eval", "N": 2048, "V": 151936, "D": 2048},
        # A toy head: four requests, where launches cost more than arithmetic.
        {"name": "ce_train_small", "op": "ce_train", "N": 64, "V": 1024, "D": 128},
        # Ragged in every direction: tokens, vocabulary and width fill no tile.
        {"name": "ce_train_ragged", "op": "ce_train", "N": 777, "V": 32003, "D": 1000},
        # A training micro-batch of 32 requests of 16 positions.
        {"name": "ce_train_32_requests", "op": "ce_train", "N": 512, "V": 151936, "D": 2048},
        # A training batch of 128 requests of 16 positions on a wide head.
        {"name": "ce_train_128_requests", "op": "ce_train", "N": 2048, "V": 151936, "D": 4096},
        # One short request in single precision: latency.
        {"name": "opd_grad_small", "op": "opd_grad", "B": 1, "k": 4, "V": 1024, "dtype": "f32"},
        # Rows of odd length, single precision.
        {"name": "opd_grad_odd", "op": "opd_grad", "B": 5, "k": 7, "V": 50021, "dtype": "f32"},
        # The whole serving batch: 128 requests, up to 16 verified positions each.
        {"name": "opd_grad_128_requests", "op": "opd_grad", "B": 128, "k": 16, "V": 151936,
         "dtype": "bf16"},
        # A few small tensors: launch latency.
        {"name": "clip_small", "op": "clip", "tensors": 12, "total": 20000, "f32_share": 0.5},
        # All layers of a drafter: hundreds of tensors, norm vectors among matrices.
        {"name": "clip_layers", "op": "clip", "tensors": 290, "total": 60000000, "f32_share": 0.3},
        # A drafter with its vocabulary head: 0.8 G gradient entries, bf16.
        {"name": "clip_with_head", "op": "clip", "tensors": 60, "total": 800000000,
         "f32_share": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ce_eval", "ce_train", "opd_grad", "clip"])
    if op in ("ce_eval", "ce_train"):
        return {"op": op, "N": _log_int(rng, 1, 2048), "V": _log_int(rng, 100, 151936),
                "D": 8 * _log_int(rng, 8, 512)}
    if op == "opd_grad":
        return {"op": op, "B": _log_int(rng, 1, 64), "k": rng.randint(1, BLOCK),
                "V": _log_int(rng, 500, 151936), "dtype": rng.choice(["bf16", "f32"])}
    return {"op": op, "tensors": _log_int(rng, 1, 400), "total": _log_int(rng, 2000, 600000000),
            "f32_share": rng.choice([0.0, 0.3, 1.0])}


def _tensor_sizes(case):
    """(entries, dtype) of each gradient tensor: sizes spread over four decades, as norm
    vectors, projections and heads are; the same for every seed of a case."""
    rng = random.Random(1000 * case["tensors"] + case["total"])
    share = [math.exp(rng.uniform(0.0, 9.0)) for _ in range(case["tensors"])]
    whole = sum(share)
    return [(max(1, int(case["total"] * s / whole)),
             torch.float32 if rng.random() < case["f32_share"] else torch.bfloat16)
            for s in share]


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _prepare_ce(case, seed):
    N, V, D = case["N"], case["V"], case["D"]
    g = _generator(seed)
    # Rows of the head have norm 2, hidden states unit entries: logits of
    # standard deviation 2; half the tokens are well predicted (their hidden
    # state leans towards their label's row), the rest are not.
    w = torch.empty((V, D), dtype=torch.bfloat16, device=DEV).normal_(
        0.0, 2.0 / math.sqrt(D), generator=g)
    labels = torch.randint(0, V, (N,), generator=g, device=DEV)
    lean = 3.0 * (torch.rand((N, 1), generator=g, device=DEV) < 0.5)
    h = torch.randn((N, D), generator=g, device=DEV) + lean * w[labels].float()
    # One token in eight carries no label (padding of a packed batch).
    skip = torch.rand(N, generator=g, device=DEV) < 0.125
    skip[0] = False
    labels = torch.where(skip, -1, labels).to(torch.int32)
    # Weights that fall with the position in its block, normalised to one.
    pos = torch.arange(N, device=DEV) % BLOCK
    tw = torch.exp(-pos.float() / 7.0) * ~skip
    s = {"hidden": h.to(torch.bfloat16), "weight": w, "labels": labels,
         "grad_nll": (tw / tw.sum()).float()}
    if own:
        import speculative_decoding_verification_58_gb300 as sv
        s["head"] = sv.LinearCe(s["hidden"], s["weight"], s["labels"],
                                s["grad_nll"] if case["op"] == "ce_train" else None)
    return s


def _prepare_opd(case, seed):
    B, k, V = case["B"], case["k"], case["V"]
    g = _generator(seed)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    target = torch.empty((B, k + 1, V), dtype=dt, device=DEV)
    draft = torch.empty((B, k, V), dtype=dt, device=DEV)
    # Zipf logits over a permutation of the vocabulary per request; the draft
    # is the target with noise.
    tail = -1.1 * torch.log(torch.arange(1, V + 1, device=DEV, dtype=torch.float32))
    for b in range(B):
        bias = tail[torch.randperm(V, generator=g, device=DEV)]
        z = torch.randn((k + 1, V), generator=g, device=DEV) + bias
        sigma = 0.3 if b % 2 == 0 else 2.0
        target[b] = z
        draft[b] = z[:k] + sigma * torch.randn((k, V), generator=g, device=DEV)
    lengths = torch.randint(1, k + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    return {"target": target, "draft": draft, "lengths": lengths,
            "grad_loss": torch.rand(B, generator=g, device=DEV) / B,
            "d_draft": torch.empty_like(draft) if own else None}


def _views(flat, sizes):
    """The tensors of a case as views into one buffer per dtype, each at a 16-byte boundary."""
    at = {dt: 0 for dt in flat}
    views = []
    for n, dt in sizes:
        views.append(flat[dt][at[dt]:at[dt] + n])
        at[dt] += -(-n // 8) * 8
    return views


def _prepare_clip(case, seed):
    g = _generator(seed)
    sizes = _tensor_sizes(case)
    length = {dt: sum(-(-n // 8) * 8 for n, d in sizes if d == dt)
              for dt in (torch.bfloat16, torch.float32)}
    flat = {dt: torch.zeros(n, dtype=dt, device=DEV) for dt, n in length.items() if n}
    out = {dt: torch.zeros_like(t) for dt, t in flat.items()}
    grads = _views(flat, sizes)
    # Gradients of different layers have different scales.
    for t in grads:
        t.normal_(0.0, 10.0 ** (-1.0 - 3.0 * float(torch.rand((), generator=g, device=DEV)))
                  if case["tensors"] < 64 else 0.01, generator=g)
    s = {"grads": grads, "out": _views(out, sizes), "flat_out": out, "max_norm": 1.0}
    if own:
        import speculative_decoding_verification_58_gb300 as sv
        s["clipper"] = sv.GradClipper(grads, s["max_norm"], out=s["out"])
    return s


def prepare(case, seed):
    op = case["op"]
    s = (_prepare_clip if op == "clip" else _prepare_opd if op == "opd_grad" else _prepare_ce)(
        case, seed)
    s["op"] = op
    return s


def _plain_ce(s):
    h, w, y = s["hidden"].float(), s["weight"].float(), s["labels"].long()
    z = h @ w.t()
    m = z.amax(1)
    lse = m + torch.log(torch.exp(z - m[:, None]).sum(1))
    has = y >= 0
    at = y.clamp(min=0)[:, None]
    nll = torch.where(has, lse - z.gather(1, at)[:, 0], 0.0)
    if s["op"] == "ce_eval":
        return nll, lse
    # z becomes the gradient of the logits in place.
    z = z.sub_(lse[:, None]).exp_()
    z.scatter_add_(1, at, torch.full_like(at, -1, dtype=z.dtype))
    z.mul_(torch.where(has, s["grad_nll"], 0.0)[:, None])
    return nll, lse, (z @ w).to(torch.bfloat16), (z.t() @ h).to(torch.bfloat16)


def _plain_opd(s):
    k = s["draft"].shape[1]
    zt, zd, L = s["target"][:, :k].float(), s["draft"].float(), s["lengths"].long()
    top = zt.argmax(2, keepdim=True)
    zt = zt - zt.amax(2, keepdim=True)
    zt = zt - torch.log(torch.exp(zt).sum(2, keepdim=True))
    zd = zd - zd.amax(2, keepdim=True)
    zd = zd - torch.log(torch.exp(zd).sum(2, keepdim=True))
    q = torch.exp(zd)
    t = zd - zt
    # An entry counts while it lies below the clip; above, its sum term is constant.
    u = torch.where(q * t < DELTA, t + 1.0, 0.0)
    grad = (1.0 - ALPHA) * q * (u - (q * u).sum(2, keepdim=True)) + ALPHA * q
    grad.scatter_add_(2, top, torch.full_like(top, -1, dtype=grad.dtype) * ALPHA)
    pos = torch.arange(k, device=L.device)[None, :]
    scale = torch.where(pos < L[:, None], s["grad_loss"][:, None] / L[:, None].float(), 0.0)
    return (grad * scale[:, :, None]).to(s["draft"].dtype)


def _plain_clip(s):
    total = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum()
    norm = total.sqrt()
    scale = (s["max_norm"] / norm).clamp(max=1.0).float()
    [o.copy_(t.float() * scale) for t, o in zip(s["grads"], s["out"])]
    return [norm.float()] + [s["flat_out"][dt] for dt in sorted(s["flat_out"], key=str)]


def run(state):
    op = state["op"]
    if not own:
        return {"opd_grad": _plain_opd, "clip": _plain_clip}.get(op, _plain_ce)(state)
    import speculative_decoding_verification_58_gb300 as sv
    if op == "ce_eval":
        return state["head"].loss()
    if op == "ce_train":
        return state["head"].loss() + state["head"].grad()
    if op == "opd_grad":
        return sv.spec_opd_grad(state["target"], state["draft"], state["lengths"],
                                state["grad_loss"], delta=DELTA, alpha=ALPHA,
                                d_draft=state["d_draft"])
    norm = state["clipper"]().reshape(())
    return [norm] + [state["flat_out"][dt] for dt in sorted(state["flat_out"], key=str)]


def work(case):
    op = case["op"]
    if op in ("ce_eval", "ce_train"):
        N, V, D = case["N"], case["V"], case["D"]
        once = 2 * N * D + 2 * V * D
        if op == "ce_eval":
            return {"bytes": once + 12 * N, "flops": 2 * N * V * D}
        return {"bytes": 2 * once + 16 * N, "flops": 6 * N * V * D}
    if op == "opd_grad":
        B, k, V = case["B"], case["k"], case["V"]
        es = 4 if case["dtype"] == "f32" else 2
        # Lengths are uniform in 1..k: (k + 1) / 2 verified positions a request.
        rows = B * (k + 1) / 2
        return {"bytes": es * V * (2 * rows + B * k) + 8 * B, "flops": 20 * rows * V}
    size = sum(n * (4 if dt == torch.float32 else 2) for n, dt in _tensor_sizes(case))
    entries = sum(n for n, _ in _tensor_sizes(case))
    return {"bytes": 2 * size + 4, "flops": 3 * entries}


def _exact_ce(case, s):
    if 6.0 * case["N"] * case["V"] * case["D"] > 9e12:  # double precision runs at about 1 TFLOP/s
        return None
    w = s["weight"].double()
    y = s["labels"].long()
    nll, lse, dh = [], [], []
    dw = torch.zeros_like(w) if case["op"] == "ce_train" else None
    for r in range(0, case["N"], 512):  # 512 rows of logits at a time
        h = s["hidden"][r:r + 512].double()
        z = h @ w.t()
        ll = torch.logsumexp(z, 1)
        lab = y[r:r + 512]
        one = torch.zeros_like(z)
        rows = torch.nonzero(lab >= 0)[:, 0]
        one[rows, lab[rows]] = 1.0
        nll.append(torch.where(lab >= 0, ll - (z * one).sum(1), 0.0))
        lse.append(ll)
        if dw is not None:
            dz = (torch.softmax(z, 1) - one) * torch.where(
                lab >= 0, s["grad_nll"][r:r + 512].double(), 0.0)[:, None]
            dh.append(dz @ w)
            dw += dz.t() @ h
    head = (torch.cat(nll), torch.cat(lse))
    return head if dw is None else head + (torch.cat(dh), dw)


def _exact_opd(case, s):
    out = torch.zeros(s["draft"].shape, dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        L = int(s["lengths"][b])
        zt = s["target"][b, :L].double()
        logp = torch.log_softmax(zt, 1)
        logq = torch.log_softmax(s["draft"][b, :L].double(), 1)
        q = logq.exp()
        term = q * (logq - logp)
        # d term_v / d logq_v, zero where the clip holds the term constant.
        slope = torch.where(term < DELTA, q + term, torch.zeros_like(q)) * (1.0 - ALPHA)
        slope[torch.arange(L, device=DEV), zt.argmax(1)] -= ALPHA
        # Through logq_v = z_v - logsumexp(z).
        out[b, :L] = (slope - q * slope.sum(1, keepdim=True)) * (
            s["grad_loss"][b].double() / L)
    return out


def _exact_clip(case, s):
    ss = [float(torch.dot(t.double(), t.double())) for t in s["grads"]]
    norm = math.sqrt(math.fsum(ss))
    f = min(1.0, s["max_norm"] / norm)
    res = {dt: torch.zeros(t.numel(), dtype=torch.float64, device=DEV)
           for dt, t in s["flat_out"].items()}
    for t, o in zip(s["grads"], _views(res, _tensor_sizes(case))):
        o.copy_(t.double() * f)
    return [torch.tensor(norm, dtype=torch.float64)] + [res[dt] for dt in sorted(res, key=str)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        return _exact_clip(case, s)
    return _exact_opd(case, s) if case["op"] == "opd_grad" else _exact_ce(case, s)
