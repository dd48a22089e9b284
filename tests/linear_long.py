"""Linear attention over long sequences in float64, 64 rows at a time, and how
far fp32 sums may be from it.  Written from the formulas of
include/gdn_linear.h in products of torch's, on any device; held to the
row-by-row oracle by test_linear_long_oracle.py."""
from __future__ import annotations

import math

import torch

ROUND = 2.0 ** -24  # half a step of fp32


def turned(t):
    return t.transpose(-1, -2).contiguous()


def attend(q, k, v, g, S, scale):
    """One sequence: q, k [rows][h][dk], v [rows][h][dv], g [rows][h] (no more
    than a few hundred a chunk below zero), S [h][dk][dv].  (o, last state)"""
    o = torch.empty_like(v)
    for r in range(0, len(q), 64):
        a, b, c = (t[r:r + 64].transpose(0, 1).contiguous() for t in (q, k, v))
        G = g[r:r + 64].cumsum(0).T.contiguous()  # [h][rows]
        D = torch.exp(torch.where(torch.ones(G.shape[1], G.shape[1], dtype=torch.bool, device=G.device).tril(),
                                  G[:, :, None] - G[:, None], -math.inf))
        o[r:r + 64] = (scale * (torch.exp(G)[..., None] * (a @ S) + (D * (a @ turned(b))) @ c)).transpose(0, 1)
        S = torch.exp(G[:, -1])[:, None, None] * S + turned(b * torch.exp(G[:, -1:] - G)[..., None]) @ c
    return o, S


def gradients(q, k, v, g, S0, scale, d_o, d_state):
    """(dq, dk, dv, dg, d_state0) of one sequence, by value head.  dq is attend
    with (d_o, v, k) for (q, k, v); dk and dv it with rows and decays turned
    round, d_state in front; dg by <S_t, E_t> written from either side."""
    dq, last = attend(d_o, v, k, g, turned(S0), scale)
    late = torch.cat((torch.zeros_like(g[:1]), g[1:].flip(0)))
    dk, _ = attend(v.flip(0), scale * d_o.flip(0), q.flip(0), late, turned(d_state), 1.0)
    dv, first = attend(k.flip(0), scale * q.flip(0), d_o.flip(0), late, d_state, 1.0)
    dk, dv = dk.flip(0), dv.flip(0)
    behind = (turned(last) * d_state).sum((1, 2))
    dg = behind + ((q * dq).sum(-1) - (k * dk).sum(-1)).flip(0).cumsum(0).flip(0)
    return dq, dk, dv, dg, torch.exp(g[0])[:, None, None] * first


def squares(q, k, v, g, S0, scale, d_o, d_state):
    """The same of the squares: the sums of squares r^2 of every result's terms."""
    o2, S2 = attend(q ** 2, k ** 2, v ** 2, 2 * g, S0 ** 2, scale ** 2)
    dq2, dk2, dv2, _, d02 = gradients(q ** 2, k ** 2, v ** 2, 2 * g, S0 ** 2, scale ** 2, d_o ** 2, d_state ** 2)
    return o2, S2, dq2, dk2, dv2, d02


def slack(dk, dv, rows):
    """fp32 sums of terms of random signs and root sum of squares r: n roundings
    of partial sums of up to 3 r, n^(1/2) 2^-24 * 3 r at random.  n: products over
    both head dims, 64 rows of a chunk, 16 for decays, and four a chunk for as
    many chunks as a state is carried."""
    return 3 * ROUND * math.sqrt(2 * max(dk, dv) + 80 + 4 * -(-rows // 64))


def state_slack(rows):
    """A state alone: 64 products a chunk, 16 for decays, four a chunk of roundings
    at its own size; no more than r, n^(1/2) 2^-24 r at random.  The decayed rows
    held in 16 bits would be off by 2^-17 / 3^(1/2) of every term at random."""
    return ROUND * math.sqrt(80 + 4 * -(-rows // 64))


def dg_error(q, k, dq2, dk2, d, whole=False):
    """The root mean square error to expect of dg of one sequence, [rows][h]:
    from row t on the terms q.dq - k.dk of every row behind, each with the error
    d times its own root sum of squares; whole: of the sum over the rows, where
    the term of row i counts i + 1 times, [h]."""
    term2 = (q ** 2 * dq2).sum(-1) + (k ** 2 * dk2).sum(-1)
    if whole:
        at = torch.arange(1, len(q) + 1, dtype=torch.float64, device=q.device)[:, None]
        return d * (at ** 2 * term2).sum(0).sqrt()
    return d * term2.flip(0).cumsum(0).flip(0).sqrt()
