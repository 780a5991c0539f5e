"""Plain double-precision forms of the drafter-training operators (test infrastructure only)."""

import torch


def ce(h, w, labels):
    """(nll, lse) in double precision."""
    z = h.double() @ w.double().t()
    lse = torch.logsumexp(z, 1)
    y = labels.long()
    has = (y >= 0) & (y < w.shape[0])
    at = torch.where(has, y, torch.zeros_like(y))
    nll = torch.where(has, lse - z.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    nll[y >= w.shape[0]] = float("nan")
    return nll, lse


def ce_grad(h, w, labels, g):
    """(d_hidden, d_weight, dZ, |g| (p + [v = y])) in double precision."""
    h, w, g = h.double(), w.double(), g.double()
    y = labels.long()
    has = (y >= 0) & (y < w.shape[0])
    p = torch.softmax(h @ w.t(), 1)
    one = torch.zeros_like(p)
    rows = torch.nonzero(has)[:, 0]
    one[rows, y[rows]] = 1.0
    gg = torch.where(has, g, torch.zeros_like(g))[:, None]
    dz = gg * (p - one)
    return dz @ w, dz.t() @ h, dz, gg.abs() * (p + one)


def opd_loss(zt, zd, lengths, delta, alpha):
    """Mixture loss [B] from target [B, k+1, V] and draft [B, k, V] in double precision."""
    out = []
    for b in range(zd.shape[0]):
        L = int(lengths[b])
        t, d = zt[b, :L].double(), zd[b, :L].double()
        lp, lq = torch.log_softmax(t, 1), torch.log_softmax(d, 1)
        q = lq.exp()
        f = torch.where(q > 0, q * (lq - lp), torch.zeros_like(q))
        hard = -lq.gather(1, t.argmax(1, keepdim=True))[:, 0]
        out.append(alpha * hard.mean() + (1 - alpha) * f.clamp(max=delta).sum(1).mean())
    return torch.stack(out)


def opd_grad(zt, zd, lengths, g, delta, alpha, flip=0.0):
    """(d_draft, per-entry error scale, log q, rows with an entry at the clip) in double precision.

    The scale of an entry is g / L q ((1 - alpha) (|u| + 1 + sum q |u|) + alpha),
    the magnitude of everything that is added up in it.  ``flip``: entries
    whose q t is within this relative distance of delta take the other side
    of the clip (at most one in a row), where the gradient jumps.
    """
    B, k, V = zd.shape
    out = torch.zeros((B, k, V), dtype=torch.float64, device=zd.device)
    scale, logq = torch.zeros_like(out), torch.zeros_like(out)
    at_clip = torch.zeros((B, k), dtype=torch.bool, device=zd.device)
    for b in range(B):
        L = int(lengths[b])
        if L < 1 or L > k:
            out[b] = float("nan")
            continue
        t, d = zt[b, :L].double(), zd[b, :L].double()
        good = torch.isfinite(torch.logsumexp(t, 1)) & torch.isfinite(torch.logsumexp(d, 1))
        lp, lq = torch.log_softmax(t, 1), torch.log_softmax(d, 1)
        q = lq.exp()
        tt = lq - lp
        f = q * tt
        below = f < delta
        near = (f / delta - 1).abs() <= flip
        if flip:
            assert int(near[good].sum(1).max() if good.any() else 0) <= 1
            below = below ^ near
            at_clip[b, :L] = near.any(1)
        u = torch.where(below, tt + 1.0, torch.zeros_like(q))
        u[q == 0] = 0.0
        s = (q * u).sum(1, keepdim=True)
        one = torch.zeros_like(q)
        one[torch.arange(L, device=q.device), t.argmax(1)] = 1.0
        y = alpha * (q - one) + (1 - alpha) * q * (u - s)
        y[~good] = float("nan")
        gl = float(g[b]) / L
        out[b, :L] = gl * y
        scale[b, :L] = abs(gl) * (q * ((1 - alpha) * (u.abs() + 1 + (q * u.abs()).sum(1, keepdim=True))
                                       + alpha) + alpha * one)
        logq[b, :L] = torch.where(q > 0, lq, torch.zeros_like(q))
    return out, scale, logq, at_clip


def norm(grads):
    """Global norm in double precision (host float); entries scaled so that no square overflows."""
    big = max([float(t.double().abs().max()) for t in grads if t.numel()] + [0.0])
    if not (0.0 < big < float("inf")):
        return big
    return big * sum(float((t.double() / big).square().sum()) for t in grads) ** 0.5
