"""The paged attention in 64 bits with a bound for every value by itself.

u = 2^-24.  One natural logit x of an fp32 evaluation is off by at most
    dx = u ((sqrt(d) + 11) size + 30),   size = max over the keys of beta sum |q k|
(a sum of d products of random signs: sqrt(d) steps of size; the scale's and the
product's rounding and the subtraction of the reference: a few of size; 2^x: 2^-22;
each rescaling, one for every 2^8 that the maximum grows: 6 u).  A sum over n
keys adds at most ds = u (sqrt(n) + 64): additions of random signs, and three
chained tensor-core products of 16 keys, which cut off up to 17 u each, and the
joins.  Numerator and normaliser each are off by dx + ds of their absolute sums.
"""

from __future__ import annotations

import math

import torch

U = 2.0 ** -24


def attend(case, coreset=None, scale=None):
    """dict of out, lse, wts (as cache_ref.attend's) and their bounds out_b, lse_b, wts_b."""
    beta = scale or 1.0 / math.sqrt(case.d)
    G = case.hq // case.hkv
    f64 = dict(dtype=torch.float64)
    r = dict(out=torch.zeros(case.B, case.hq, case.dv, **f64), out_b=torch.zeros(case.B, case.hq, case.dv, **f64),
             lse=torch.full((case.B, case.hq), -math.inf, **f64), lse_b=torch.zeros(case.B, case.hq, **f64),
             wts=torch.zeros(case.B, case.hkv, case.cap, **f64), wts_b=torch.zeros(case.B, case.hkv, case.cap, **f64))
    for b in range(case.B):
        for h in range(case.hkv):
            k, v = case.rows(b, h)
            n = k.shape[0]
            ext = torch.cat([v, torch.ones(n, 1, **f64)], 1)
            if coreset is not None:
                Ks, W, rank = coreset
                m = Ks.shape[2] if rank is None else int(rank[b, h])
                k = torch.cat([k, Ks[b, h, :m].double()])
                ext = torch.cat([ext, W[b, h, :m].double()])
            if k.shape[0] == 0:
                continue
            g = slice(h * G, (h + 1) * G)
            q = case.q[b, g].double()
            x = beta * q @ k.T
            size = (beta * q.abs() @ k.abs().T).amax(1, keepdim=True)
            dx = U * ((math.sqrt(case.d) + 11) * size + 30)
            ds = U * (math.sqrt(k.shape[0]) + 64)
            top = x.amax(1, keepdim=True)
            a = torch.exp(x - top)
            A, S = a @ ext, a @ ext.abs()
            L, spread = A[:, -1:], S[:, -1:] / A[:, -1:].abs()
            r["out"][b, g] = A[:, :-1] / L
            r["out_b"][b, g] = (dx + ds) * (S[:, :-1] / L.abs() + spread * (A[:, :-1] / L).abs()) + U * (A[:, :-1] / L).abs()
            r["lse"][b, g] = (top + torch.log(L))[:, 0]
            r["lse_b"][b, g] = ((dx + ds) * spread)[:, 0] + U * r["lse"][b, g].abs()
            w = a[:, :n] / L
            r["wts"][b, h, :n] = w.sum(0)
            old = case.scores[b, h, :n].double().abs()
            r["wts_b"][b, h, :n] = ((dx + (dx + ds) * spread + 4 * U) * w).sum(0) + U * (old + 2 * G * w.sum(0))
    return r


def check(got, want, bound, what):
    """Each value within its bound (and a value of -inf equal to it)."""
    got = got.cpu().double()
    same = got == want
    off = torch.where(same, torch.zeros_like(got), (got - want).abs() - bound)
    assert torch.isfinite(off).all() and float(off.max()) <= 0, (what, float(off.max()), int(off.argmax()))
