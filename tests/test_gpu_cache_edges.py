"""The paged cache on the GPU at its edges: what the calls promise for refused
sequences, extreme values, other streams and rows outside the cache."""

import math
import types

import pytest
import torch

import cache_bounds
import cache_ref
from coreset_attention_approximation_b200 import wildcat
from parity import TOL_OUT, rel_err

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def test_evict_into_refuses_a_few_of_many():
    """More blocks than the GPU holds at once, thousands of kept rows, and a
    few sequences refused for each reason: those stay as they are, and every
    other one is moved."""
    B, hkv, page, d, n, keep = 64, 8, 16, 8, 3000, 2500
    g = torch.Generator().manual_seed(1)
    m = -(-n // page)
    order = torch.randperm(2 * B * m, generator=g).to(torch.int32)
    table, into = order[: B * m].reshape(B, m).clone(), order[B * m:].reshape(B, m).clone()
    k0 = torch.randn(2 * B * m, hkv, page, d, generator=g).to(BF)
    v0 = torch.randn(2 * B * m, hkv, page, d, generator=g).to(BF)
    s0 = torch.rand(B, hkv, m * page, generator=g)
    used = -(-keep // page)
    into[3, used - 1] = 2 * B * m                # no page
    into[17, 5] = into[18, 6]                    # one page for two sequences
    into[40, 0] = into[40, 1]                    # and for two places of one
    into[41, 2] = table[7, 9]                    # a page that is read
    table[63, m - 1] = -9                        # no page among those read
    refused = [3, 17, 18, 40, 41, 63]
    lens = torch.full((B,), n, dtype=torch.int32)
    k, v, scores = k0.cuda(), v0.cuda(), s0.cuda()
    to = torch.full_like(scores, -7.0)
    cache = wildcat.PagedCache(k, v, table.cuda(), hq=hkv, scores=scores)
    res = cache.evict(lens.cuda(), keep, sink=4, recent=64, into=into.cuda(), scores_into=to)
    assert cache.check() in (1, 7)               # (the first that was recorded)
    idx, new = res["idx"].cpu(), res["lens"].tolist()
    want_k, want_v, want_s = k0.clone(), v0.clone(), torch.full_like(s0, -7.0)
    at = torch.arange(keep)
    for b in range(B):
        assert new[b] == (n if b in refused else keep)
        if b in refused:
            assert torch.all(idx[b] == -1)
            continue
        for h in range(hkv):
            src = torch.from_numpy(cache_ref.kept_positions(s0[b, h].numpy(), n, keep, 4, 64))
            assert torch.equal(idx[b, h].long(), src)
            f, t = table[b].long()[src // page], into[b].long()[at // page]
            want_k[t, h, at % page], want_v[t, h, at % page] = k0[f, h, src % page], v0[f, h, src % page]
            want_s[b, h, :keep] = s0[b, h, src]
    assert torch.equal(k.cpu(), want_k) and torch.equal(v.cpu(), want_v) and torch.equal(to.cpu(), want_s)
    assert torch.equal(scores.cpu(), s0)


ROOM = pytest.mark.parametrize("room", [1, 16])   # short tables (one launch) and long ones (divided and joined)


@ROOM
@pytest.mark.parametrize("dtype,group", [(BF, 1), (BF, 4), (BF, 7), (BF, 8), (BF, 16), (BF, 20), (F32, 3), (F32, 16)])
@pytest.mark.parametrize("equal", [False, True])
def test_attend_infinite_values(dtype, group, equal, room):
    """An infinite value makes its column infinite for the queries of its kv
    head (both infinities, or a NaN: NaN), and changes no bit of anything else.
    With equal keys every weight is exact in 8 bits."""
    case = cache_ref.Case(dtype, 3, 2 * group, 2, 64, 48, 16, 20 * room, [300, 77, 16], seed=group)
    if equal:
        case.k[~torch.isnan(case.k)] = 0.25

    def run():
        k, v, table, q, lens, _ = case.on_gpu()
        cache = wildcat.PagedCache(k, v, table, hq=2 * group)
        out = cache.attend(q, lens)
        assert cache.check() == 0
        return out.cpu()

    clean = run()
    assert torch.isfinite(clean).all()
    inf, at = float("inf"), lambda b, t: (int(case.table[b, t // 16]), 1, t % 16)      # kv head 1
    case.v[at(0, 3)][0] = inf
    case.v[at(0, 299)][47] = inf
    case.v[at(0, 200)][9] = -inf
    case.v[at(0, 17)][30], case.v[at(0, 170)][30] = inf, -inf
    case.v[at(0, 40)][31] = float("nan")
    case.v[at(2, 15)][5], case.v[at(2, 0)][5] = -inf, -inf
    got = run()
    want = clean.clone()
    heads = slice(group, 2 * group)
    want[0, heads, 0], want[0, heads, 47], want[0, heads, 9], want[2, heads, 5] = inf, inf, -inf, -inf
    want[0, heads, 30] = want[0, heads, 31] = float("nan")
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, nan=0.5, posinf=inf, neginf=-inf),
                       torch.nan_to_num(want, nan=0.5, posinf=inf, neginf=-inf))


@ROOM
@pytest.mark.parametrize("dtype,group", [(BF, 2), (BF, 8), (BF, 16), (F32, 1), (F32, 4), (F32, 8)])
@pytest.mark.parametrize("r", [0, 200])
def test_attend_huge_values(dtype, group, r, room):
    """Values about 2^121 and logits that rise by 5 behind the first tiles of a
    warp: no product may overflow, in the pages or in a coreset.  600 sequences
    with the same pages, so that every warp has several tiles."""
    B, n, d = 600, 300, 64
    case = cache_ref.Case(dtype, 1, group, 1, d, d, 16, 20 * room, [n], seed=3)
    case.k = 0.125 * torch.round(case.k.float())                   # (unused slots stay NaN)
    for t in range(n):
        case.k[int(case.table[0, t // 16]), 0, t % 16, 0] = 0.0 if t < 64 else 5.0
    case.k = case.k.to(dtype)
    case.q[..., 0] = 8.0                                           # beta <q, k> = k[0] + noise
    case.v = (case.v.float() * 2.0 ** 120).to(dtype)
    core = None
    if r:
        g = torch.Generator().manual_seed(5)
        Ks = 0.125 * torch.round(torch.randn(1, 1, r, d, generator=g))
        Ks[..., 0] = 5.0 * (torch.arange(r) // 32 % 2)
        w = 1.0 + torch.rand(1, 1, r, 1, generator=g)
        core = (Ks.to(dtype), torch.cat([w * torch.randn(1, 1, r, d, generator=g) * 2.0 ** 120, w], -1), None)
    many = lambda x: x.cuda().expand(B, *x.shape[1:]).contiguous()
    cache = wildcat.PagedCache(case.k.cuda(), case.v.cuda(), many(case.table), hq=group, scores=many(case.scores))
    out, lse = cache.attend(many(case.q), many(case.lens), coreset=core and (many(core[0]), many(core[1]), None),
                            accumulate=True, return_lse=True)
    assert cache.check() == 0
    ref = cache_bounds.attend(case, core)
    cache_bounds.check(out, ref["out"], ref["out_b"], "out")
    cache_bounds.check(lse, ref["lse"], ref["lse_b"], "lse")
    cache_bounds.check(cache.scores.cpu().double() - case.scores.double(), ref["wts"], ref["wts_b"], "scores")


def small_cache(B=2, n_pages=16, hkv=2, page=16, d=64, hq=4):
    k, v = (torch.randn(n_pages, hkv, page, d, device="cuda").to(BF) for _ in range(2))
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda").reshape(B, -1)
    scores = torch.rand(B, hkv, table.shape[1] * page, device="cuda")
    return wildcat.PagedCache(k, v, table, hq=hq, scores=scores)


def test_a_stream_of_another_device_is_refused():
    """Also the default stream, whose handle is the same on every device."""
    cache = small_cache()
    other = types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=torch.cuda.default_stream().cuda_stream)
    K = torch.ones(2, 2, 1, 64, dtype=BF, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    before = cache.k_pages.clone()
    with pytest.raises(wildcat.WildcatError, match="another device"):
        cache.append(K, K, pos, stream=other)
    assert torch.equal(cache.k_pages, before)


def test_first_call_on_another_stream():
    """Made behind long work on one stream, in memory that was used before,
    and called at once on another: the workspace is ready."""
    cache = small_cache()
    k, v, table, scores = cache.k_pages, cache.v_pages, cache.table, cache.scores
    lens = torch.tensor([100, 128], dtype=torch.int32, device="cuda")
    want = cache.evict(lens, 40, into=table, scores_into=torch.zeros_like(scores))["idx"].cpu()
    n = cache.ws.numel()
    del cache
    torch.full((n,), 255, dtype=torch.uint8, device="cuda")       # (freed at once)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                                 # about a tenth of a second
    cache = wildcat.PagedCache(k, v, table, hq=4, scores=scores)
    with torch.cuda.stream(side):
        res = cache.evict(lens, 40)
    side.synchronize()
    assert cache.check() == 0 and torch.equal(res["idx"].cpu(), want) and res["lens"].tolist() == [40, 40]


def test_the_workspace_outlives_its_cache_on_another_stream():
    """A cache dropped while another stream still runs its calls: the
    workspace's memory is not given to anyone before they are done."""
    cache = small_cache()
    at = cache.ws.data_ptr()
    side = torch.cuda.Stream()
    q = torch.randn(2, 4, 64, device="cuda").to(BF)
    lens = torch.tensor([100, 128], dtype=torch.int32, device="cuda")
    cache.attend(q, lens, accumulate=True)                         # (a kernel's first launch may wait for the GPU)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)
        out = cache.attend(q, lens, accumulate=True)
    del cache
    blocks = [x for seg in torch.cuda.memory_snapshot() for x in seg["blocks"] if x["address"] == at]
    assert not side.query()
    assert [x["state"] for x in blocks] == ["active_pending_free"]
    side.synchronize()
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("kw", [{}, {"center": True}, {"bins": 4}, {"bins": 4, "center": True}])
def test_compressed_prompt_and_exact_tail_are_one_softmax(dtype, kw):
    """A prompt of 5 distinct keys a bin, which its coreset reproduces exactly,
    and a tail in the pages: exact attention over all tokens, in value and in
    normaliser.  The coreset's share is as far off as the library's attention
    over it alone may be (its tolerance), and the joint row is no further."""
    B, hq, hkv, n, d, r, tail = 2, 8, 2, 1024, 64, 64, [90, 7]
    g = torch.Generator().manual_seed(6)
    distinct = torch.randn(B, hkv, 4, 1, 5, d, generator=g, dtype=torch.float64) * 0.6
    K = distinct.expand(B, hkv, 4, 52, 5, d).reshape(B, hkv, 4, 260, d)[:, :, :, :256].reshape(B, hkv, n, d).to(dtype)
    if kw.get("center"):
        K = (K.double() + 0.4).to(dtype)
    V = torch.randn(B, hkv, n, d, generator=g, dtype=torch.float64).to(dtype)
    case = cache_ref.Case(dtype, B, hq, hkv, d, d, 16, 8, tail, seed=9, key_scale=0.6)
    case.q = (0.6 * case.q.double()).to(dtype)
    sel = wildcat.select(K.cuda(), r, seed=5, **kw)
    wts = wildcat.weights(K.cuda(), V.cuda(), sel["piv"], sel["F"], sel["rank"], r, **kw)
    k, v, table, q, lens, _ = case.on_gpu()
    cache = wildcat.PagedCache(k, v, table, hq=hq)
    out, lse = cache.attend(q, lens, coreset=(wts["Ks"], wts["W"], sel["rank"]), return_lse=True)
    assert cache.check() == 0
    for b in range(B):
        for h in range(hkv):
            kk, vv = case.rows(b, h)
            kk, vv = torch.cat([K[b, h].double(), kk]), torch.cat([V[b, h].double(), vv])
            x = case.q[b, 4 * h:4 * h + 4].double() @ kk.T / 8.0
            want = torch.softmax(x, -1) @ vv
            assert rel_err(out[b, 4 * h:4 * h + 4].cpu(), want) <= TOL_OUT[dtype]
            off = (lse[b, 4 * h:4 * h + 4].cpu().double() - torch.logsumexp(x, -1)).abs().max()
            assert float(off) <= TOL_OUT[dtype]


def test_ranks_of_bins_are_checked():
    cache = small_cache()
    q = torch.ones(2, 4, 64, dtype=BF, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    Ks, W = torch.ones(2, 2, 8, 64, dtype=BF, device="cuda"), torch.ones(2, 2, 8, 65, device="cuda")
    for rank in (torch.ones(2, 2, 3), torch.ones(2, 2, 0), torch.ones(2, 1, 4), torch.ones(2, 2, 4).double()):
        rank = rank.cuda() if rank.dtype == torch.double else rank.to(torch.int32).cuda()
        with pytest.raises(wildcat.WildcatError):
            cache.attend(q, lens, coreset=(Ks, W, rank))
    out = cache.attend(q, lens, coreset=(Ks, W, torch.full((2, 2, 4), 2, dtype=torch.int32, device="cuda")))
    assert torch.equal(out, torch.ones_like(out))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_writes_the_rows_inside_and_no_other(dtype):
    """Positions and counts outside the cache, a page outside the pool: the
    rows whose place is inside land there, whole, and everything else (pages,
    scores) keeps its bits."""
    B, hkv, page, t, d, dv = 3, 2, 16, 4, 64, 40
    case = cache_ref.Case(dtype, B, hkv, hkv, d, dv, page, 4, [64] * B, seed=14)
    k, v, table, _, _, scores = case.on_gpu()
    cache = wildcat.PagedCache(k, v, table, hq=hkv, scores=scores)
    bad = case.table.clone()
    bad[2, 1] = case.n_pages
    want_k, want_v, want_s = case.k.clone(), case.v.clone(), case.scores.clone()
    same = lambda x, y: torch.equal(torch.nan_to_num(x.cpu().float(), nan=9e9), torch.nan_to_num(y.float(), nan=9e9))
    g = torch.Generator().manual_seed(2)
    for i, (pos, count, tab) in enumerate([
            ([62, 0, 5], [4, 0, 2], case.table), ([-2, 7, 60], [4, 4, 4], case.table),
            ([0, 8, 9], [-1, 9, 1], case.table), ([2 ** 31 - 2, 63, -2 ** 31], [4, 1, 4], case.table),
            ([64, 64, 14], [1, 4, 4], bad), ([20, 21, 30], None, bad), ([-4, -3, 61], None, case.table)]):
        K = torch.randn(B, hkv, t, d, generator=g).to(dtype)
        V = torch.randn(B, hkv, t, dv, generator=g).to(dtype)
        outside = False
        for b in range(B):
            n = t if count is None else count[b]
            outside |= not 0 <= n <= t
            for j in range(min(max(n, 0), t)):
                at = pos[b] + j
                p = int(tab[b, at // page]) if 0 <= at < 64 else -1
                if not 0 <= p < case.n_pages:
                    outside = True
                    continue
                want_k[p, :, at % page], want_v[p, :, at % page], want_s[b, :, at] = K[b, :, j], V[b, :, j], 0.0
        cache.table.copy_(tab)
        cache.append(K.cuda(), V.cuda(), torch.tensor(pos, dtype=torch.int32).cuda(),
                     None if count is None else torch.tensor(count, dtype=torch.int32).cuda())
        assert cache.check() == (7 if outside else 0), i
        assert same(cache.k_pages, want_k) and same(cache.v_pages, want_v), i
        assert torch.equal(cache.scores.cpu(), want_s), i


def ones_of(case):
    """The case with every value that is there 1: each output is a row's sum of
    weights over its normaliser."""
    case.v = torch.where(torch.isnan(case.v), case.v, torch.ones_like(case.v))
    return case


@ROOM
@pytest.mark.parametrize("group", [1, 4, 5, 8, 9, 16, 17])
def test_attend_value_product_keeps_all_bits_of_the_weights(group, room):
    """bf16 values of 1: out = (sum of the weights' three terms) / (sum of the
    weights), whatever 2^x rounds to.  Of the numerator, each 16-key product cuts
    off up to 17 u (u = 2^-24) three times over, at most 3 x 17 u; it and the
    normaliser each take a rounding for each of at most 19 + 3 additions in a
    warp, 19 in a join and its factors, and the quotient one: (51 + 2 x 42) u =
    135 u = 8e-6.  A second term is some thousandths of its weight."""
    case = ones_of(cache_ref.Case(BF, 3, 2 * group, 2, 64, 64, 16, 20 * room, [300, 130, 16], seed=group))
    k, v, table, q, lens, _ = case.on_gpu()
    cache = wildcat.PagedCache(k, v, table, hq=2 * group)
    out = cache.attend(q, lens).cpu().double()
    assert cache.check() == 0
    assert float((out - 1).abs().max()) <= 135 * cache_bounds.U
    # and each column its own: a power of two each, exact in every step
    scale = (2.0 ** torch.arange(-32, 32).float()).to(BF)
    cache.v_pages.mul_(scale.cuda())
    assert torch.equal(cache.attend(q, lens).cpu().double(), out * scale.double())


@ROOM
@pytest.mark.parametrize("group", [1, 2, 4, 7, 8, 13, 16])
def test_attend_value_product_keeps_the_last_bits_of_the_weights(group, room):
    """The same with one key of logit 0 and all others of a logit whose weight
    beside it is t / 2, t = 1 + 2^-8 + 200 2^-23: its third term is 200 2^-23 (a
    few units more or less, as 2^x and the scale round), 2.4e-5 of it and three
    times the bound.  Every second query row is 0: weights of exactly 2^-8, whose
    second and third terms are nothing, so another row's terms would show too."""
    t = 1 + 2.0 ** -8 + 200 * 2.0 ** -23
    case = ones_of(cache_ref.Case(BF, 2, group, 1, 64, 64, 16, 20 * room, [300, 40], seed=group))
    live = ~torch.isnan(case.k)
    case.k = torch.where(live, torch.zeros_like(case.k), case.k)
    case.k[..., 0] = torch.where(live[..., 0], -torch.ones_like(case.k[..., 0]), case.k[..., 0])
    for b in range(2):
        case.k[int(case.table[b, 0]), 0, 0, 0] = 0
    case.q.zero_()
    case.q[:, ::2, 0] = 1
    k, v, table, q, lens, _ = case.on_gpu()
    cache = wildcat.PagedCache(k, v, table, hq=group, scale=math.log(2.0) * (1 - math.log2(t)))
    out, lse = cache.attend(q, lens, return_lse=True)
    assert cache.check() == 0
    n = case.lens.double()[:, None]
    want = torch.log(torch.where(torch.arange(group) % 2 == 0, 1 + (n - 1) * t / 2, n))
    assert float((lse.cpu().double() - want).abs().max()) <= 64 * cache_bounds.U      # the case is the one meant
    assert float((out.cpu().double() - 1).abs().max()) <= 135 * cache_bounds.U


@pytest.mark.parametrize("group", [4, 8, 16])
def test_attend_does_not_drift_over_long_stretches(group):
    """512 sequences over the same 65536 keys with values of 1, hundreds of
    steps a warp: roundings to nearest average out over the rows, so the mean
    output is 1 up to what each 16-key product cuts off (3 x 17 u at most) and
    the join's and the quotient's few; sums kept by the tensor core itself would
    lose part of an u at every step, all one way."""
    n, B, d = 65536, 512, 16
    case = ones_of(cache_ref.Case(BF, 1, group, 1, d, d, 4096, 16, [n], seed=group))
    g = torch.Generator().manual_seed(1)
    q = torch.randn(B, group, d, generator=g).to(BF).cuda()
    table = case.table.cuda().expand(B, -1).contiguous()
    cache = wildcat.PagedCache(case.k.cuda(), case.v.cuda(), table, hq=group)
    out = cache.attend(q, torch.full((B,), n, dtype=torch.int32, device="cuda")).double()
    assert cache.check() == 0
    assert abs(float(out.mean()) - 1) <= (51 + 9) * cache_bounds.U
    # one row: 2 x 900 steps' roundings of random signs, of which the largest of a few thousand is 5 deviations
    # of sqrt(1800 / 3) u each, beside the 60 u
    assert float((out - 1).abs().max()) <= (60 + 5 * (1800 / 3) ** 0.5) * cache_bounds.U


@ROOM
@pytest.mark.parametrize("dtype,hq,hkv,d,dv,page,tf", [
    (BF, 8, 2, 128, 128, 16, False), (BF, 32, 4, 128, 128, 64, True), (BF, 16, 1, 128, 64, 32, False),
    (BF, 10, 2, 96, 96, 24, False), (BF, 24, 2, 256, 256, 7, True), (BF, 36, 1, 64, 128, 16, False),
    (F32, 8, 2, 64, 64, 16, False), (F32, 16, 1, 256, 256, 32, False), (F32, 20, 2, 40, 136, 16, False)])
@pytest.mark.parametrize("core", [0, 1, 70])
def test_attend_every_value_within_its_own_bound(dtype, hq, hkv, d, dv, page, tf, core, room):
    lens = [0, 1, 16, 65, 300]
    case = cache_ref.Case(dtype, len(lens), hq, hkv, d, dv, page, -(-304 * room // page), lens, tokens_first=tf, seed=d + core)
    cs = None
    if core:
        g = torch.Generator().manual_seed(core)
        w = torch.exp(torch.randn(case.B, hkv, core, 1, generator=g))
        cs = (torch.randn(case.B, hkv, core, d, generator=g).to(dtype),
              torch.cat([w * torch.randn(case.B, hkv, core, dv, generator=g), w], -1),
              torch.randint(0, core + 1, (case.B, hkv), generator=g).to(torch.int32))
    k, v, table, q, lens, scores = case.on_gpu()
    cache = wildcat.PagedCache(k, v, table, hq=hq, scores=scores)
    out, lse = cache.attend(q, lens, coreset=cs and tuple(x.cuda() for x in cs), accumulate=True, return_lse=True)
    assert cache.check() == 0
    ref = cache_bounds.attend(case, cs)
    cache_bounds.check(out, ref["out"], ref["out_b"], "out")
    cache_bounds.check(lse, ref["lse"], ref["lse_b"], "lse")
    cache_bounds.check(cache.scores.cpu().double() - case.scores.double(), ref["wts"], ref["wts_b"], "scores")
