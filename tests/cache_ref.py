"""Plain 64-bit forms of the paged cache's operators (CPU, torch fp64 and
loops), the random caches that the tests feed both sides, and the error bound
of an fp32 attention."""

from __future__ import annotations

import math

import numpy as np
import torch


class Case:
    """A cache with random pages, every sequence's pages drawn without
    repetition.  Slots that no token uses hold NaN, table entries that no token
    uses hold a number that is no page: neither may be read."""

    def __init__(self, dtype, B, hq, hkv, d, dv, page, max_pages, lens, tokens_first=False, seed=0, key_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.hq, self.hkv, self.d, self.dv, self.page = B, hq, hkv, d, dv, page
        self.max_pages, self.cap, self.dtype = max_pages, max_pages * page, dtype
        self.tokens_first = tokens_first
        self.n_pages = B * max_pages + 2
        self.table = torch.randperm(self.n_pages, generator=g)[: B * max_pages].reshape(B, max_pages).to(torch.int32)
        self.k = (key_scale * torch.randn(self.n_pages, hkv, page, d, generator=g)).to(dtype)
        self.v = torch.randn(self.n_pages, hkv, page, dv, generator=g).to(dtype)
        self.q = torch.randn(B, hq, d, generator=g).to(dtype)
        self.scores = torch.rand(B, hkv, self.cap, generator=g)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.hide_unused()

    def hide_unused(self):
        used = torch.zeros(self.n_pages, self.page, dtype=torch.bool)
        for b in range(self.B):
            n = int(self.lens[b])
            for t in range(n):
                used[int(self.table[b, t // self.page]), t % self.page] = True
            self.table[b, (n + self.page - 1) // self.page:] = -5
        keep = used[:, None, :, None]
        self.k = torch.where(keep, self.k, torch.full_like(self.k, float("nan")))
        self.v = torch.where(keep, self.v, torch.full_like(self.v, float("nan")))

    def on_gpu(self):
        """(k, v, table, q, lens, scores) on the GPU, the pools in the case's order."""
        def pool(x):
            x = x.cuda()
            return x.transpose(1, 2).contiguous().transpose(1, 2) if self.tokens_first else x

        return (pool(self.k), pool(self.v), self.table.cuda(), self.q.cuda(), self.lens.cuda(), self.scores.cuda())

    def rows(self, b, h, n=None):
        """Keys and values of sequence b, kv head h in 64 bits."""
        n = int(self.lens[b]) if n is None else n
        t = torch.arange(n)
        pages = self.table[b].long()[t // self.page]
        return self.k[pages, h, t % self.page].double(), self.v[pages, h, t % self.page].double()


def attend(case, coreset=None, scale=None):
    """(out, lse, weights [B, Hkv, cap], bound): the definition in 64 bits and
    how far an fp32 evaluation may be off, per output value of unit |v|."""
    beta = scale or 1.0 / math.sqrt(case.d)
    G = case.hq // case.hkv
    out = torch.zeros(case.B, case.hq, case.dv, dtype=torch.float64)
    lse = torch.full((case.B, case.hq), -math.inf, dtype=torch.float64)
    wts = torch.zeros(case.B, case.hkv, case.cap, dtype=torch.float64)
    worst = 0.0
    for b in range(case.B):
        for h in range(case.hkv):
            k, v = case.rows(b, h)
            n = k.shape[0]
            ext = torch.cat([v, torch.ones(n, 1, dtype=torch.float64)], 1)
            keys = k
            if coreset is not None:
                Ks, W, rank = coreset
                r = Ks.shape[2] if rank is None else int(rank[b, h])
                keys = torch.cat([k, Ks[b, h, :r].double()])
                ext = torch.cat([ext, W[b, h, :r].double()])
            if keys.shape[0] == 0:
                continue
            for g in range(h * G, (h + 1) * G):
                q = case.q[b, g].double()
                x = beta * (keys @ q)
                top = x.max()
                a = torch.exp(x - top)
                A = a @ ext
                out[b, g] = A[:-1] / A[-1]
                lse[b, g] = top + torch.log(A[-1])
                wts[b, h, :n] += a[:n] / A[-1]
                # rounding of a logit: sums of d products (random signs: sqrt(d) steps) of sum |q k|, its
                # scaling and the subtraction of the maximum; of the sums over n keys: sqrt(n) steps; of
                # 2^x, the quotient and the joins: a few.  Twice that, times the weights' absolute sum.
                size = float((beta * (keys.abs() @ q.abs())).max())
                cancel = float((a @ ext.abs()).max() / A[-1].abs())
                worst = max(worst, 2 * 2.0 ** -24 * ((math.sqrt(case.d) + 4) * size + math.sqrt(keys.shape[0]) + 16)
                            * max(cancel, 1.0))
    return out, lse, wts, worst


def kept_positions(scores, n, keep, sink, recent):
    """Ascending kept positions of one row of scores with n tokens."""
    if n <= keep:
        return np.arange(n)
    x = np.array(scores[:n], dtype=np.float64)
    x[np.isnan(x)] = -np.inf
    middle = np.arange(sink, n - recent)
    order = middle[np.argsort(-x[middle] + 0.0, kind="stable")]
    want = keep - sink - recent
    return np.sort(np.concatenate([np.arange(sink), order[:want], np.arange(n - recent, n)]).astype(np.int64))
