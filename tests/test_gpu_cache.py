"""The paged cache on the GPU against its plain 64-bit forms: append, attention
of one new token (with and without a coreset), eviction, and a run of them
together."""

import math

import numpy as np
import pytest
import torch

import cache_ref
from cache_ref import Case
from coreset_attention_approximation_b200 import wildcat

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(case, scores=True, **kw):
    k, v, table, q, lens, sc = case.on_gpu()
    cache = wildcat.PagedCache(k, v, table, hq=case.hq, scores=sc if scores else None, **kw)
    return cache, q, lens


def plain(pages):
    """Values with a number in the place of each NaN (unused slots, NaN scores)."""
    return torch.nan_to_num(pages.cpu().float(), nan=9e9)


def check_attend(case, coreset=None, accumulate=True, scale=0.0):
    cache, q, lens = make(case, scores=accumulate, scale=scale)
    cs = None if coreset is None else tuple(None if t is None else t.cuda() for t in coreset)
    out, lse = cache.attend(q, lens, coreset=cs, accumulate=accumulate, return_lse=True)
    assert cache.check() == 0
    want, wlse, wts, bound = cache_ref.attend(case, coreset, scale or None)
    vmax = float(torch.nan_to_num(case.v.float()).abs().max())
    if coreset is not None:     # the ratio of W's columns to its last one plays the values' part
        vmax = max(vmax, 1.0)
    assert out.dtype == F32
    out, lse = out.cpu().double(), lse.cpu().double()
    empty = wlse == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert torch.all(out[empty] == 0)
    err = float((out - want).abs().max()) if want.numel() else 0.0
    assert err <= bound * vmax, (err, bound * vmax)
    if not torch.all(empty):
        elog = (lse - wlse)[~empty].abs().max()
        # lse itself is rounded to fp32
        assert float(elog) <= bound + 2.0 ** -24 * float(wlse[~empty].abs().max()), (float(elog), bound)
    if accumulate:
        got = cache.scores.cpu().double()
        old = case.scores.double()
        for b in range(case.B):
            n = int(case.lens[b])
            assert torch.equal(got[b, :, n:], old[b, :, n:])
            G = case.hq // case.hkv
            if n:
                lim = bound * G + 2.0 ** -24 * (float(old.max()) + G)
                assert float((got - old - wts)[b, :, :n].abs().max()) <= lim
    return err


SHAPES = [
    # dtype, hq, hkv, d, dv, page, tokens_first
    (BF, 8, 2, 128, 128, 16, False),
    (BF, 32, 8, 128, 128, 64, True),
    (BF, 4, 4, 64, 64, 16, True),
    (BF, 16, 1, 128, 64, 32, False),
    (BF, 10, 2, 96, 96, 24, False),
    (BF, 24, 2, 256, 256, 7, True),
    (BF, 3, 3, 72, 40, 1, False),
    (BF, 36, 1, 64, 128, 16, False),
    (BF, 2, 1, 8, 16, 16, False),
    (F32, 8, 2, 64, 64, 16, False),
    (F32, 4, 4, 128, 128, 24, True),
    (F32, 16, 1, 256, 256, 32, False),
    (F32, 6, 2, 8, 8, 5, True),
    (F32, 20, 2, 40, 136, 16, False),
    (BF, 80, 1, 64, 64, 16, False),
    (F32, 70, 1, 16, 16, 16, False),
]


# Tables of this many times the tokens: short ones take a block for each head,
# long ones the division of all tiles and the join.
ROOM = pytest.mark.parametrize("room", [1, 16])


@ROOM
@pytest.mark.parametrize("dtype,hq,hkv,d,dv,page,tf", SHAPES)
def test_attend_shapes(dtype, hq, hkv, d, dv, page, tf, room):
    """Head layouts, widths, page sizes and orders; lengths of 0, 1, about a
    tile's and a page's end, and several tiles."""
    lens = [0, 1, 15, 16, 17, 63, 64, 65, 130, 300]
    case = Case(dtype, len(lens), hq, hkv, d, dv, page, -(-304 * room // page), lens, tokens_first=tf, seed=hq + d)
    check_attend(case)


@pytest.mark.parametrize("dtype,dv,n", [(BF, 64, 384), (BF, 128, 385), (BF, 256, 576), (F32, 64, 192), (F32, 64, 193)])
def test_attend_full_tables_about_the_short_ones_end(dtype, dv, n):
    case = Case(dtype, 1, 4, 2, 64, dv, 1, n, [n], seed=n)
    check_attend(case)


def test_attend_many_short_heads():
    """A table that is short for many heads only."""
    case = Case(BF, 80, 4, 4, 16, 16, 32, 16, [(37 * i) % 513 for i in range(80)], seed=29)
    check_attend(case)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[1], [5000], [0, 0, 0], [9001, 3, 0, 700], [0] * 70 + [33] + [0] * 70,
                                  [2, 1] * 150])
def test_attend_lengths(dtype, lens):
    """One sequence and many; one long among short ones; none with tokens."""
    case = Case(dtype, len(lens), 4, 2, 64, 64, 32, -(-max(max(lens), 32) // 32), lens, seed=len(lens))
    check_attend(case)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_thousands_of_sequences(dtype):
    """More sequences than a block holds places for."""
    lens = [(7 * i) % 23 if i % 5 else 0 for i in range(2500)] + [90] + [0] * 30
    case = Case(dtype, len(lens), 2, 1, 16, 16, 8, 12, lens, seed=24)
    check_attend(case)


def test_attend_in_tables_far_longer_than_the_sequences():
    """Room for 2^20 tokens, some of it used: positions beyond what one round
    of the score blocks takes, and none of it elsewhere."""
    page, n = 4096, 90000
    case = Case(BF, 1, 2, 1, 16, 16, page, 22, [n], seed=27)
    k, v, table, q, lens, _ = case.on_gpu()
    wide = torch.full((600, 256), -1, dtype=torch.int32)
    wide[7, :22] = case.table[0]
    q600 = torch.zeros(600, 2, 16, dtype=BF, device="cuda")
    q600[7] = q[0]
    l600 = torch.zeros(600, dtype=torch.int32, device="cuda")
    l600[7] = n
    cache = wildcat.PagedCache(k, v, wide.cuda(), hq=2, scores=torch.zeros(600, 1, 256 * page, device="cuda"))
    out = cache.attend(q600, l600, accumulate=True)
    assert cache.check() == 0
    want, _, wts, bound = cache_ref.attend(case)
    assert float((out[7].cpu().double() - want[0]).abs().max()) <= bound * 6
    assert float((cache.scores[7, 0, :n].cpu().double() - wts[0, 0, :n]).abs().max()) <= 2 * bound
    cache.scores[7, 0, :n] = 0
    assert not cache.scores.any() and not out[:7].any() and not out[8:].any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_without_scores_and_lse(dtype):
    case = Case(dtype, 3, 8, 2, 64, 64, 16, 40, [640, 100, 0], seed=5)
    check_attend(case, accumulate=False)
    cache, q, lens = make(case, scores=False)
    a = cache.attend(q, lens)
    b, _ = cache.attend(q, lens, return_lse=True)
    c = cache.attend(q, lens, out=torch.empty_like(a))
    assert torch.equal(a, b) and torch.equal(a, c)


def test_attend_scale_and_repeat():
    case = Case(BF, 2, 8, 2, 128, 128, 16, 128, [2000, 900], seed=6)
    check_attend(case, scale=0.03)
    cache, q, lens = make(case, scores=False)
    assert torch.equal(cache.attend(q, lens), cache.attend(q, lens))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_peaked_rows(dtype):
    """Logits over hundreds: the maximum moves along the keys, most weights
    underflow, none overflow."""
    case = Case(dtype, 2, 4, 2, 64, 64, 16, 80, [1200, 77], seed=7, key_scale=40.0)
    check_attend(case)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_equal_keys_average_the_values(dtype):
    case = Case(dtype, 1, 2, 1, 64, 64, 16, 40, [600], seed=8)
    case.k[~torch.isnan(case.k)] = 0.25
    check_attend(case)


def coreset_of(case, r, seed, full_rank=True):
    g = torch.Generator().manual_seed(seed)
    Ks = torch.randn(case.B, case.hkv, r, case.d, generator=g).to(case.dtype)
    w = torch.exp(torch.randn(case.B, case.hkv, r, 1, generator=g))
    W = torch.cat([w * torch.randn(case.B, case.hkv, r, case.dv, generator=g), w], -1).contiguous()
    rank = torch.randint(0, r + 1, (case.B, case.hkv), generator=g).to(torch.int32)
    if full_rank:
        rank[:] = r
    else:
        rank[0, 0] = 0
    return Ks, W, rank


@pytest.mark.parametrize("dtype,hq,hkv,d,dv,r", [(BF, 32, 8, 128, 128, 200), (BF, 4, 4, 64, 64, 1),
                                                 (BF, 12, 1, 96, 40, 65), (F32, 8, 2, 64, 64, 300),
                                                 (F32, 16, 1, 256, 256, 33), (BF, 2, 1, 256, 256, 1000),
                                                 (BF, 36, 1, 64, 64, 70), (F32, 20, 1, 40, 8, 9), (BF, 4, 2, 256, 8, 33),
                                                 (F32, 2, 2, 8, 136, 12), (BF, 16, 2, 8, 256, 130)])
@pytest.mark.parametrize("full", [True, False])
def test_attend_with_a_coreset(dtype, hq, hkv, d, dv, r, full):
    """One softmax over the coreset and the pages; sequences without tokens
    (the coreset alone), and ranks of 0 (the pages alone, or nothing)."""
    case = Case(dtype, 4, hq, hkv, d, dv, 16, 20, [0, 1, 100, 320], seed=r)
    check_attend(case, coreset=coreset_of(case, r, r, full))


def test_attend_with_every_row_of_a_coreset():
    case = Case(F32, 2, 4, 2, 64, 64, 16, 20, [0, 320], seed=3)
    Ks, W, _ = coreset_of(case, 40, 1)
    check_attend(case, coreset=(Ks, W, None))


def test_attend_coreset_alone_equals_attend():
    """A cache without tokens and a coreset from the library's own selection:
    the same as wildcat.attend, within the fp32 path's tolerance."""
    g = torch.Generator().manual_seed(4)
    B, hq, hkv, n, d, dv, r = 2, 4, 2, 700, 64, 64, 48
    K = (0.3 * torch.randn(B, hkv, n, d, generator=g)).cuda()
    V = torch.randn(B, hkv, n, dv, generator=g).cuda()
    Q = torch.randn(B, hq, 1, d, generator=g).cuda()
    res = wildcat.forward(Q, K, V, r, seed=1)
    case = Case(F32, B, hq, hkv, d, dv, 16, 2, [0] * B, seed=9)
    cache, _, lens = make(case)
    out = cache.attend(Q[:, :, 0], lens, coreset=(res["Ks"], res["W"], res["rank"]))
    want = res["out"][:, :, 0]
    assert float((out - want).abs().max() / want.abs().max()) <= 1e-5


@ROOM
def test_attend_infinite_and_nan_inputs_stay_in_their_rows(room):
    """A NaN query row gives NaN there and nowhere else; -inf logits weigh 0."""
    case = Case(F32, 2, 4, 2, 64, 64, 16, 20 * room, [300, 200], seed=10)
    case.q[0, 1, 3] = float("nan")
    page, slot = int(case.table[1, 2]), 5
    case.k[page, 0, slot] = -float("inf")
    case.q[1, :2] = case.q[1, :2].abs() + 0.1       # kv head 0's queries: <q, k> = -inf at that key
    cache, q, lens = make(case)
    out = cache.attend(q, lens).cpu()
    assert torch.isnan(out[0, 1]).all()
    ok = torch.ones(2, 4, dtype=torch.bool)
    ok[0, 1] = False
    case.q[0, 1] = 0
    case.k[page, 0, slot] = -1e30
    want, _, _, bound = cache_ref.attend(case)
    del bound                                        # (it counts the huge key); the others' rows are ordinary
    assert float((out.double() - want)[ok].abs().max()) <= 1e-5


@ROOM
def test_attend_rows_that_are_all_minus_infinity(room):
    case = Case(F32, 1, 1, 1, 8, 8, 16, 20 * room, [20], seed=11)
    case.q[:] = 1.0
    case.k[~torch.isnan(case.k)] = -float("inf")
    cache, q, lens = make(case)
    out, lse = cache.attend(q, lens, return_lse=True, accumulate=True)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)
    assert torch.equal(cache.scores.cpu(), case.scores)


@ROOM
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_strided_queries(dtype, room):
    """Queries as a slice of a projection's output, at an odd offset."""
    case = Case(dtype, 3, 8, 2, 64, 64, 16, 20 * room, [320, 7, 0], seed=12)
    cache, q, lens = make(case)
    wide = torch.zeros(3, 8, 64 + 11, dtype=dtype, device="cuda")
    wide[..., 3:67] = q
    assert torch.equal(cache.attend(wide[..., 3:67], lens), cache.attend(q, lens))


@ROOM
def test_attend_bad_pages_and_lengths_are_reported_and_left_out(room):
    case = Case(BF, 3, 8, 2, 64, 64, 16, 20 * room, [320, 100, 50], seed=13)
    cache, q, lens = make(case)
    good = cache.attend(q, lens)
    table = case.table.clone()
    table[1, 2] = case.n_pages
    cache.table.copy_(table)
    out = cache.attend(q, lens)
    assert cache.check() == 7 and cache.check() == 0
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    # sequence 1 without tokens 32..47
    ref = Case(BF, 3, 8, 2, 64, 64, 16, 20 * room, [320, 100, 50], seed=13)
    k, v = [], []
    for h in range(2):
        kk, vv = ref.rows(1, h)
        keep = torch.ones(100, dtype=torch.bool)
        keep[32:48] = False
        k.append(kk[keep]), v.append(vv[keep])
    for g in range(8):
        x = (k[g // 4] @ ref.q[1, g].double()) / 8.0
        want = torch.softmax(x, 0) @ v[g // 4]
        assert float((out[1, g].cpu().double() - want).abs().max()) <= 1e-5
    cache.table.copy_(case.table)
    bad = lens.clone()
    bad[2] = -4
    out = cache.attend(q, bad)
    assert cache.check() == 7
    assert torch.all(out[2] == 0) and torch.equal(out[:2], good[:2])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tf", [False, True])
@pytest.mark.parametrize("page,t", [(16, 1), (7, 40), (1, 5), (64, 3)])
def test_append(dtype, tf, page, t):
    """Rows land where the table says, scores there are cleared, nothing else
    moves; counts of 0, ragged counts and positions inside a page."""
    B, hkv, d, dv = 4, 3, 72, 40
    cap = 120
    case = Case(dtype, B, hkv, hkv, d, dv, page, -(-cap // page), [cap - page + 1] * B, tokens_first=tf, seed=t)
    cache, _, _ = make(case)
    g = torch.Generator().manual_seed(t)
    K = torch.randn(B, t, hkv, d + 8, generator=g).to(dtype).cuda().transpose(1, 2)[..., 8:]     # strided
    V = torch.randn(B, hkv, t, dv, generator=g).to(dtype).cuda()
    pos = torch.tensor([0, 3, 17, cap - page - t], dtype=torch.int32)
    count = torch.tensor([t, 0, min(t, 2), t], dtype=torch.int32)
    k, v, sc = case.k.clone(), case.v.clone(), case.scores.clone()
    for use in (count, None):
        for b in range(B):
            for j in range(t if use is None else int(count[b])):
                at = int(pos[b]) + j
                p, s = int(case.table[b, at // page]), at % page
                k[p, :, s], v[p, :, s], sc[b, :, at] = K[b, :, j].cpu(), V[b, :, j].cpu(), 0.0
        cache.append(K, V, pos.cuda(), count=None if use is None else use.cuda())
        assert cache.check() == 0
        assert torch.equal(plain(cache.k_pages), plain(k)) and torch.equal(plain(cache.v_pages), plain(v))
        assert torch.equal(cache.scores.cpu(), sc)


def test_append_outside_is_reported_and_not_written():
    case = Case(BF, 3, 2, 2, 64, 64, 16, 4, [64, 64, 64], seed=14)
    cache, _, _ = make(case)
    K = torch.ones(3, 2, 4, 64, dtype=BF, device="cuda")
    for pos, count in (([62, 0, 0], [4, 0, 0]), ([-2, 0, 0], [4, 0, 0]), ([0, 0, 0], [0, -1, 0]),
                       ([2 ** 31 - 2, 0, 0], [4, 0, 0]), ([0, 0, 0], [0, 9, 0])):
        before = plain(cache.k_pages)
        cache.append(K, K, torch.tensor(pos, dtype=torch.int32).cuda(), torch.tensor(count, dtype=torch.int32).cuda())
        assert cache.check() == 7
        changed = (plain(cache.k_pages) != before).any(dim=-1)
        inside = sum(1 for j in range(min(count[0], 4)) if 0 <= pos[0] + j < 64) + min(max(count[1], 0), 4)
        assert int(changed.sum()) <= inside * 2
    table = case.table.clone()
    table[0, 0] = -1
    cache.table.copy_(table)
    before = plain(cache.k_pages)
    zero = torch.zeros(3, dtype=torch.int32).cuda()
    cache.append(2 * K, K, zero, torch.tensor([4, 0, 0], dtype=torch.int32).cuda())
    assert cache.check() == 7 and torch.equal(plain(cache.k_pages), before)
    cache.append(K[:, :, :0], K[:, :, :0], zero)
    assert cache.check() == 0


def evict_reference(case, keep, sink, recent):
    """(idx, new lens) of every (sequence, kv head)."""
    idx = -np.ones((case.B, case.hkv, keep), dtype=np.int64)
    for b in range(case.B):
        n = int(case.lens[b])
        for h in range(case.hkv):
            p = cache_ref.kept_positions(case.scores[b, h].numpy(), n, keep, sink, recent)
            idx[b, h, : len(p)] = p
    return idx, np.minimum(case.lens.numpy(), keep)


def check_evict(case, keep, sink, recent, into, own_scores):
    cache, _, lens = make(case)
    k0, v0, s0 = cache.k_pages.clone(), cache.v_pages.clone(), cache.scores.clone()
    kw = {}
    target = case.table
    if into:
        # pages of its own behind the others
        k = torch.cat([cache.k_pages, torch.zeros_like(cache.k_pages)])
        v = torch.cat([cache.v_pages, torch.zeros_like(cache.v_pages)])
        target = torch.arange(case.B * case.max_pages, dtype=torch.int32).reshape(case.B, -1) + case.n_pages
        cache = wildcat.PagedCache(k, v, cache.table, hq=case.hq, scores=cache.scores)
        k0, v0 = k.clone(), v.clone()
        kw["into"] = target.cuda()
    if own_scores:
        kw["scores_into"] = torch.full_like(s0, -7.0)
    res = cache.evict(lens, keep, sink=sink, recent=recent, **kw)
    assert cache.check() == 0
    idx, new = evict_reference(case, keep, sink, recent)
    assert np.array_equal(res["lens"].cpu().numpy(), new)
    assert np.array_equal(res["idx"].cpu().numpy(), idx)
    k, v = k0.cpu().clone(), v0.cpu().clone()
    old_k, old_v = k.clone(), v.clone()
    s = kw["scores_into"].cpu() * 0 - 7.0 if own_scores else s0.cpu().clone()
    for b in range(case.B):
        moves = into or int(case.lens[b]) > keep
        for h in range(case.hkv):
            src = torch.from_numpy(idx[b, h, : new[b]])
            at = torch.arange(int(new[b]))
            s[b, h, at] = s0.cpu()[b, h, src]
            if moves:
                f, t = case.table[b].long()[src // case.page], target[b].long()[at // case.page]
                k[t, h, at % case.page] = old_k[f, h, src % case.page]
                v[t, h, at % case.page] = old_v[f, h, src % case.page]
    assert torch.equal(plain(cache.k_pages), plain(k)) and torch.equal(plain(cache.v_pages), plain(v))
    assert torch.equal(plain(kw["scores_into"] if own_scores else cache.scores), plain(s))


@pytest.mark.parametrize("dtype,d,dv,page,tf", [(BF, 128, 128, 16, False), (F32, 64, 40, 7, True), (BF, 8, 256, 1, False),
                                                (F32, 256, 256, 64, True)])
@pytest.mark.parametrize("keep,sink,recent", [(50, 4, 10), (1, 0, 0), (1, 1, 0), (8, 3, 5), (300, 0, 0), (64, 0, 64),
                                              (999, 16, 100)])
@pytest.mark.parametrize("into,own_scores", [(False, False), (True, True)])
def test_evict(dtype, d, dv, page, tf, keep, sink, recent, into, own_scores):
    lens = [1100, 0, 1, 50, 51, 301, 777]
    case = Case(dtype, len(lens), 2, 2, d, dv, page, -(-1100 // page), lens, tokens_first=tf, seed=keep)
    case.scores[0, 0] = 0.5                                     # all equal: the lower positions
    case.scores[6, 1, ::3] = float("nan")
    case.scores[6, 0] = torch.round(case.scores[6, 0] * 8) - 4  # many ties, both signs, zeros
    case.scores[6, 0, 5::7] *= -0.0
    check_evict(case, keep, sink, recent, into, own_scores)


@pytest.mark.parametrize("into,own_scores", [(True, False), (False, True)])
def test_evict_one_side_in_place(into, own_scores):
    lens = [400, 20, 90]
    case = Case(BF, 3, 4, 2, 64, 64, 16, 25, lens, seed=15)
    check_evict(case, 60, 2, 8, into, own_scores)


@pytest.mark.parametrize("n", [20000, 70001])
def test_evict_long(n):
    case = Case(BF, 1, 2, 2, 8, 8, 256, -(-n // 256), [n], seed=16)
    case.scores[0, 0] = torch.exp(3 * torch.randn(case.cap))
    case.scores[0, 1, 100:] = 0.0
    check_evict(case, 9000, 4, 500, False, False)


def test_evict_more_than_is_held():
    """Stretches of positions that a block cannot hold: many (sequence, kv
    head) pairs, one of them long."""
    g = torch.Generator().manual_seed(28)
    B, n, page, keep = 200, 30000, 1000, 700
    table = torch.full((B, 31), -1, dtype=torch.int32)
    table[3, :30] = torch.randperm(31, generator=g)[:30].to(torch.int32)
    k = torch.randn(31, 1, page, 8, generator=g).to(BF).cuda()
    scores = torch.rand(B, 1, 31 * page, generator=g)
    scores[3, 0, ::3] = 0.75
    lens = torch.zeros(B, dtype=torch.int32)
    lens[3] = n
    cache = wildcat.PagedCache(k, k.clone(), table.cuda(), hq=1, scores=scores.cuda())
    res = cache.evict(lens.cuda(), keep, sink=5, recent=50)
    assert cache.check() == 0
    want = cache_ref.kept_positions(scores[3, 0].numpy(), n, keep, 5, 50)
    assert np.array_equal(res["idx"][3, 0].cpu().numpy(), want)
    assert int(res["lens"][3]) == keep and int(res["lens"].sum()) == keep


def test_evict_again_and_again():
    """Calls one after the other, in place (given as such, or by the table
    itself), with refusals between them: no count of pages is left over."""
    case = Case(BF, 2, 2, 2, 64, 64, 16, 30, [470, 200], seed=25)
    cache, _, lens = make(case)
    for keep, into in ((300, None), (250, cache.table), (250, None), (100, None), (99, cache.table), (3, None)):
        before = cache.scores.cpu().clone()
        n = lens.tolist()
        res = cache.evict(lens, keep, recent=2, into=into, lens_out=lens)
        assert cache.check() == 0 and lens.tolist() == [min(x, keep) for x in n]
        for b in range(2):
            for h in range(2):
                want = cache_ref.kept_positions(before[b, h].numpy(), n[b], keep, 0, 2)
                assert np.array_equal(res["idx"][b, h, : len(want)].cpu().numpy(), want)
        if keep == 250:
            good = cache.table.clone()
            cache.table[1, 0] = cache.table[0, 0]
            left = lens.tolist()
            cache.evict(lens, 20, lens_out=lens)
            assert cache.check() == 1 and lens.tolist() == left
            cache.table.copy_(good)


def test_evict_captured():
    """Captured once, replayed on restored scores: the same kept positions as
    an eager call, whichever call came before."""
    case = Case(F32, 2, 2, 2, 64, 64, 16, 30, [470, 200], seed=26)
    cache, _, lens = make(case)
    k, v, sc = cache.k_pages.clone(), cache.v_pages.clone(), cache.scores.clone()
    want = cache.evict(lens, 70, sink=1, recent=9)
    after = plain(cache.k_pages), plain(cache.v_pages), cache.scores.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.k_pages.copy_(k), cache.v_pages.copy_(v), cache.scores.copy_(sc)
        res = cache.evict(lens, 70, sink=1, recent=9)
    for i in range(4):
        graph.replay()
        assert torch.equal(res["idx"], want["idx"]) and torch.equal(res["lens"], want["lens"])
        assert torch.equal(plain(cache.k_pages), after[0]) and torch.equal(plain(cache.v_pages), after[1])
        assert torch.equal(cache.scores, after[2])
        if i == 1:
            cache.evict(lens, 300)
    assert cache.check() == 0


def test_pools_beyond_four_gigabytes():
    """Pages whose offsets pass 32 bits, in bytes and in elements: append,
    attention and eviction there."""
    page, d, n_pages, top = 65536, 128, 560, 555          # 16 MiB a page; 9 GiB of keys and 9 of values
    k = torch.empty(n_pages, 1, page, d, dtype=BF, device="cuda")
    v = torch.empty(n_pages, 1, page, d, dtype=BF, device="cuda")
    table = torch.tensor([[top, 3], [256, 400]], dtype=torch.int32, device="cuda")
    scores = torch.zeros(2, 1, 2 * page, device="cuda")
    cache = wildcat.PagedCache(k, v, table, hq=4, scores=scores)
    g = torch.Generator().manual_seed(3)
    n = 300
    K, V = (torch.randn(2, 1, n, d, generator=g).to(BF) for _ in range(2))
    Q = torch.randn(2, 4, d, generator=g).to(BF)
    pos = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    cache.append(K.cuda(), V.cuda(), pos)
    cache.append(K.cuda()[:, :, :5], V.cuda()[:, :, :5], torch.zeros_like(pos), torch.tensor([0, 5], dtype=torch.int32).cuda())
    lens = torch.tensor([n, n + 5], dtype=torch.int32, device="cuda")
    assert torch.equal(k[top, 0, :n].cpu(), K[0, 0]) and torch.equal(v[256, 0, 5:n + 5].cpu(), V[1, 0])
    out = cache.attend(Q.cuda(), lens, accumulate=True)
    for b in range(2):
        kk = K[b, 0] if b == 0 else torch.cat([K[b, 0, :5], K[b, 0]])
        vv = V[b, 0] if b == 0 else torch.cat([V[b, 0, :5], V[b, 0]])
        p = torch.softmax(Q[b].double() @ kk.double().T / math.sqrt(d), -1)
        # the fp32 bound of cache_ref.attend for these sizes: 128 products of at most 20 in all, 305 keys
        assert float((out[b].cpu().double() - p @ vv.double()).abs().max()) <= 2 ** -23 * (15.4 * 20 + 34) * 5
        res = cache.scores[b, 0, : len(kk)].cpu().double() - p.sum(0)
        assert float(res.abs().max()) <= 2 ** -23 * (15.4 * 20 + 34) * 4
    idx = cache.evict(lens, 40)["idx"].cpu().long()
    assert cache.check() == 0
    assert torch.equal(k[top, 0, :40].cpu(), K[0, 0][idx[0, 0]])
    assert torch.equal(v[256, 0, :40].cpu(), torch.cat([V[1, 0, :5], V[1, 0]])[idx[1, 0]])


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured, with nothing run before."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch
from coreset_attention_approximation_b200 import wildcat
k = torch.randn(8, 2, 16, 64, device="cuda").bfloat16()
table = torch.arange(8, dtype=torch.int32, device="cuda").reshape(2, 4)
scores = torch.zeros(2, 2, 64, device="cuda")
cache = wildcat.PagedCache(k, k.clone(), table, hq=4, scores=scores)
q = torch.randn(2, 4, 64, device="cuda").bfloat16()
new = torch.randn(2, 2, 1, 64, device="cuda").bfloat16()
lens = torch.tensor([50, 7], dtype=torch.int32, device="cuda")
core = (torch.randn(2, 2, 9, 64, device="cuda").bfloat16(), torch.rand(2, 2, 9, 65, device="cuda"), None)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    cache.append(new, new, lens)
    out = cache.attend(q, lens, coreset=core, accumulate=True)
    res = cache.evict(lens, 20)
g.replay()
torch.cuda.synchronize()
assert cache.check() == 0 and res["lens"].tolist() == [20, 7] and bool(torch.isfinite(out).all())
print("fine")
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "fine" in done.stdout, done.stderr[-2000:]


def test_evict_extreme_scores():
    case = Case(F32, 1, 1, 1, 8, 8, 16, 10, [160], seed=17)
    s = case.scores[0, 0]
    s[:] = -float("inf")
    s[10], s[20], s[30], s[40], s[50] = float("inf"), 3e38, 1e-45, -1e-45, float("nan")
    check_evict(case, 6, 0, 0, False, False)
    check_evict(case, 3, 1, 1, False, False)


def test_evict_refuses_shared_and_bad_pages():
    """A sequence whose pages cannot be written stays as it is and the others
    are served; into pages of their own the same sequences are copied."""
    def fresh():
        c = Case(BF, 3, 2, 2, 64, 64, 16, 10, [160, 160, 100], seed=18)
        c.table[1, 0] = c.table[0, 0]              # a shared first page
        cache, _, lens = make(c)
        return c, cache, lens

    case, cache, lens = fresh()
    k0, s0 = cache.k_pages.clone(), cache.scores.clone()
    res = cache.evict(lens, 40)
    assert cache.check() == 1
    assert res["lens"].tolist() == [160, 160, 40]
    assert torch.all(res["idx"][:2] == -1) and torch.all(res["idx"][2] >= 0)
    for b in (0, 1):
        pages = case.table[b].long()
        assert torch.equal(plain(cache.k_pages)[pages], plain(k0)[pages])
        assert torch.equal(cache.scores[b], s0[b])
    # into: reading shared pages is fine; a page of `into` named twice, or one of the table's, is not
    case, cache, lens = fresh()
    spare = [p for p in range(case.n_pages) if p not in set(case.table.flatten().tolist())]
    into = torch.full((3, 10), -1, dtype=torch.int32)
    into[0, :1], into[1, :1], into[2, :1] = spare[0], spare[1], spare[2]
    res = cache.evict(lens, 16, into=into.cuda())
    assert cache.check() == 0 and res["lens"].tolist() == [16, 16, 16]
    case, cache, lens = fresh()
    into[1, 0], into[2, 0] = spare[0], int(case.table[2, 3])
    res = cache.evict(lens, 16, into=into.cuda(), lens_out=lens)
    assert cache.check() == 1 and res["lens"].tolist() == [160, 160, 100] and res["lens"] is lens
    assert torch.all(res["idx"] == -1)
    # no page at all
    case, cache, lens = fresh()
    cache.table[2, 6] = case.n_pages + 3
    res = cache.evict(lens, 155)
    assert cache.check() in (1, 7) and res["lens"].tolist() == [160, 160, 100]
    case, cache, lens = fresh()
    into[0, 0], into[1, 0], into[2, 0] = spare[0], -1, spare[2]
    res = cache.evict(lens, 16, into=into.cuda())
    assert cache.check() == 7 and res["lens"].tolist() == [16, 160, 16]


@ROOM
def test_shared_pages_are_read_alike(room):
    """Two sequences with the same pages attend to the same rows, and each
    accumulates its own scores."""
    case = Case(BF, 2, 4, 2, 64, 64, 16, 10 * room, [150, 150], seed=19)
    case.table[1] = case.table[0]
    case.q[1] = case.q[0]
    cache, q, lens = make(case)
    cache.scores.zero_()
    out = cache.attend(q, lens, accumulate=True)
    assert torch.equal(out[0], out[1]) and torch.equal(cache.scores[0], cache.scores[1])


@ROOM
def test_captured_step_serves_a_growing_cache(room):
    """append, attend and the length's advance captured once, replayed over
    eight tokens: the same bits as eager calls on a copy of the cache."""
    def cache_of():
        case = Case(BF, 2, 8, 2, 64, 64, 16, 8 * room, [128, 128], seed=20)
        cache, _, _ = make(case)
        return cache, torch.tensor([30, 61], dtype=torch.int32, device="cuda")

    g = torch.Generator().manual_seed(1)
    K, V, Q = (torch.randn(8, 2, n, 64, generator=g).to(BF).cuda() for n in (2, 2, 8))
    eager, lens = cache_of()
    want = []
    for i in range(8):
        eager.append(K[i][:, :, None], V[i][:, :, None], lens)
        lens += 1
        want.append(eager.attend(Q[i], lens, accumulate=True))
    cache, lens = cache_of()
    k, v, q = (torch.zeros_like(x[0]) for x in (K, V, Q))
    start = lens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.append(k[:, :, None], v[:, :, None], lens, torch.zeros_like(lens))
        cache.attend(q, lens)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(k[:, :, None], v[:, :, None], lens)
        lens += 1
        out = cache.attend(q, lens, accumulate=True)
    lens.copy_(start)
    for i in range(8):
        k.copy_(K[i]), v.copy_(V[i]), q.copy_(Q[i])
        graph.replay()
        assert torch.equal(out, want[i]), i
    assert torch.equal(cache.scores, eager.scores) and cache.check() == 0


def test_captured_behind_copies_and_other_streams():
    """The step captured behind a copy, a memset and another stream's kernel:
    what stands before it in the graph is done when it reads."""
    case = Case(BF, 2, 8, 2, 64, 64, 16, 100, [1600, 900], seed=23)
    cache, q, lens = make(case)
    core = tuple(t.cuda() for t in coreset_of(case, 100, 5))
    plain_out = cache.attend(q, lens)
    core_out = cache.attend(q, lens, coreset=core)
    q2, lens2, big = torch.zeros_like(q), torch.zeros_like(lens), torch.randn(1 << 24, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q2.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            big.mul_(1.0)
            lens2.copy_(lens)
        q2.copy_(q)
        torch.cuda.current_stream().wait_stream(side)
        a = cache.attend(q2, lens2)
        q2.zero_()
        q2.copy_(q)
        b = cache.attend(q2, lens2, coreset=core)
        q2.zero_()
        lens2.zero_()
    for _ in range(3):
        graph.replay()
        assert torch.equal(a, plain_out) and torch.equal(b, core_out)
    # and eagerly, each call behind the one before
    for _ in range(20):
        big.mul_(1.0)
        lens2.copy_(lens)
        q2.copy_(q)
        a = cache.attend(q2, lens2)
        b = cache.attend(q2, lens2, coreset=core)
        c = cache.attend(q2, lens2)
        lens2.zero_()
        q2.zero_()
        assert torch.equal(a, plain_out) and torch.equal(b, core_out) and torch.equal(c, plain_out)


def test_other_stream():
    case = Case(BF, 4, 8, 2, 64, 64, 16, 100, [1600, 900, 0, 5], seed=21)
    cache, q, lens = make(case)
    want = cache.attend(q, lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = cache.attend(q, lens, stream=side)
    res = cache.evict(lens, 100, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and res["lens"].tolist() == [100, 100, 0, 5]


@ROOM
@pytest.mark.parametrize("dtype", [BF, F32])
def test_serving_run(dtype, room):
    """Prompt, decode steps with accumulation, eviction, more steps: against
    the same run in 64 bits (its own scores decide its evictions; the scores
    are far enough apart for both to keep the same tokens)."""
    B, hq, hkv, d, page, keep = 2, 4, 2, 64, 16, 40
    case = Case(dtype, B, hq, hkv, d, d, page, 8 * room, [128] * B, seed=22)
    case.scores.zero_()
    cache, _, _ = make(case)
    g = torch.Generator().manual_seed(2)
    lens = torch.tensor([70, 33], dtype=torch.int32)
    gl = lens.cuda()
    for step in range(24):
        K, V, Q = (torch.randn(B, n, d, generator=g).to(dtype) for n in (hkv, hkv, hq))
        cache.append(K.cuda()[:, :, None], V.cuda()[:, :, None], gl)
        for b in range(B):
            at = int(lens[b])
            p, s = int(case.table[b, at // page]), at % page
            case.k[p, :, s], case.v[p, :, s], case.scores[b, :, at] = K[b], V[b], 0.0
        gl += 1
        lens += 1
        case.lens, case.q = lens, Q
        out = cache.attend(Q.cuda(), gl, accumulate=True)
        want, _, wts, bound = cache_ref.attend(case)
        assert float((out.cpu().double() - want).abs().max()) <= bound * float(torch.nan_to_num(case.v.float()).abs().max())
        case.scores += wts.float()
        if step == 11:
            idx, new = evict_reference(case, keep, 2, 8)
            res = cache.evict(gl, keep, sink=2, recent=8, lens_out=gl)
            assert np.array_equal(res["idx"].cpu().numpy(), idx)
            k, v, sc = case.k.clone(), case.v.clone(), case.scores.clone()
            for b in range(B):
                if int(lens[b]) <= keep:
                    continue
                for h in range(hkv):
                    src, at = torch.from_numpy(idx[b, h]), torch.arange(keep)
                    f, t = case.table[b].long()[src // page], case.table[b].long()[at // page]
                    k[t, h, at % page], v[t, h, at % page] = case.k[f, h, src % page], case.v[f, h, src % page]
                    sc[b, h, :keep] = case.scores[b, h, src]
            case.k, case.v, case.scores = k, v, sc
            lens = torch.from_numpy(new.astype(np.int32))
    assert cache.check() == 0 and gl.tolist() == lens.tolist()
