"""Double-precision references of truncated sampling and of attention over a paged cache."""

import math

import torch

NEAR = 1e-9  # relative distance of a border from a sum below which either side may be taken


def _near(x, border, unit):
    """Whether a value is next to the border, but not at it (u = 0, equal logits)."""
    d = (x - border).abs()
    return bool(((d < NEAR * unit) & (d > 0)).any())


def truncate(z, T, k=0, p=1.0, m=0.0):
    """One row (any float type): (kept, masses, near).  ``near``: a border lies within NEAR."""
    z = z.double()
    V = z.numel()
    kept = torch.zeros(V, dtype=torch.bool, device=z.device)
    if T == 0.0:
        kept[int(torch.nonzero(z == z[~torch.isnan(z)].max())[0])] = True
        return kept, kept.double(), False
    w = torch.exp((z - z.max()) / T)
    order = torch.argsort(-z, stable=True)
    if k > 0:
        order = order[:k]
    near = False
    if p < 1.0:
        c = torch.cumsum(w[order], 0)
        want = p * c[-1]
        order = order[:int((c < want).sum()) + 1]
        near = _near(c, want, c[-1])
    kept[order] = True
    if m > 0.0:
        kept &= w >= m
        near = near or _near(w, m, m)
    return kept, torch.where(kept, w, 0.0), near


def draw(w, u):
    """(index, near) of the inverse CDF over masses ``w``."""
    c = torch.cumsum(w, 0)
    level = u * c[-1]
    near = _near(c, level, c[-1])
    return int((c <= level).sum()), near


def paged_entries(cache, table_row, total):
    """[total, heads, width] in double precision."""
    P = cache.shape[1]
    at = torch.arange(total, device=cache.device)
    return cache[table_row[at // P].long(), at % P].double()


def attention(q, k, v, causal, window, scale):
    """q [n, H, D], k, v [total, Hk, D], double: out [n, H, D], lse [n, H], and the sums and
    sizes that error bounds are made of: sum_j p_j |v_j| [n, H, D], max_j scale sum_d |q_d k_jd| [n, H]."""
    n, H, D = q.shape
    total, Hk = k.shape[:2]
    G = H // Hk
    out, mass = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    size = torch.zeros((n, H), dtype=torch.float64, device=q.device)
    pos = torch.arange(total - n, total, device=q.device)[:, None]
    at = torch.arange(total, device=q.device)[None, :]
    sees = torch.ones((n, total), dtype=torch.bool, device=q.device)
    if causal:
        sees = at <= pos
        if window:
            sees &= at > pos - window
    some = sees.any(1)
    if total == 0:
        return out, lse, mass, size
    for h in range(H):
        kh, vh = k[:, h // G], v[:, h // G]
        s = torch.where(sees, scale * (q[:, h] @ kh.t()), -math.inf)
        p = torch.where(some[:, None], torch.softmax(s, 1), 0.0)
        out[:, h], mass[:, h] = p @ vh, p @ vh.abs()
        lse[:, h] = torch.logsumexp(s, 1)
        size[:, h] = torch.where(sees, scale * (q[:, h].abs() @ kh.abs().t()), 0.0).amax(1)
    return out, lse, mass, size
