"""Truncated sampling in double precision, many settings of one row at a time, with how far the
library's whole-number masses may be from it.

The library's mass of an entry is a whole number of units of the largest entry's mass: off by
half a unit, and by 2^-37 of itself.  A sum of n masses out of S is therefore off by at most
2^-37 S + n / 2 units, and so is what it is compared with (a share of such a sum): `slack` is both.
"""

import torch


def unit(V):
    """The largest entry's mass is a whole number of these (2^-45, coarser where V masses would
    not fit 64 bits)."""
    return 2.0 ** -min(45, 63 - max(1, (V - 1).bit_length()))


def slack(total, n, V):
    return 2.0 ** -36 * total + n * unit(V)


def masses(z, T):
    """[..., V] of the largest entry's mass, in double precision."""
    z = z.double()
    return torch.exp((z - z.amax(-1, keepdim=True)) / T)


def draws(w, u):
    """The least and the largest index that the uniforms ``u`` [n] may draw from the masses ``w``
    [V] (0: not kept)."""
    c = torch.cumsum(w, 0)
    total = c[-1]
    s = slack(total, int((w > 0).sum()), w.numel())
    level = u.double() * total
    lo = torch.searchsorted(c, level - s, right=True)
    hi = torch.searchsorted(c, level + s, right=True)
    # (Behind the last kept entry there is nothing to draw.)
    last = int(torch.nonzero(w > 0)[-1])
    return lo.clamp(max=last), hi.clamp(max=last)


def counts(w, p):
    """How many of the masses ``w`` [V], largest first, the shares ``p`` [n] may keep: the least
    number and the largest."""
    c = torch.cumsum(w, 0)
    s = slack(c[-1], w.numel(), w.numel())
    want = p.double() * c[-1]
    lo = torch.searchsorted(c, want - s) + 1
    hi = torch.searchsorted(c, want + s) + 1
    return lo.clamp(max=w.numel()), hi.clamp(max=w.numel())


def at_borders(c, i, step=0):
    """Single-precision shares next to c[i] / c[-1], ``step`` numbers further up, below 1."""
    x = (c[i] / c[-1]).float()
    for _ in range(abs(step)):
        x = torch.nextafter(x, torch.full_like(x, 2.0 if step > 0 else -1.0))
    return x.clamp(2.0 ** -24, 1.0 - 2.0 ** -24)
