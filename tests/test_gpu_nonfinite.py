"""Infinities and NaN among what the paged attention and the paged indexer read: they reach the
results as the formulas carry them, and nothing else."""
import math

import pytest
import torch

import lightning_indexer_b200 as dsa
import paged_testutil as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
INF, NAN = float("inf"), float("nan")


def pages(Hq, Hkv, d, page, n, k, seed):
    """One sequence of n positions, k of them selected (all where k >= n), on shuffled pages."""
    g = torch.Generator().manual_seed(seed)
    width = (n + page - 1) // page
    table = torch.randperm(width, generator=g)[None].to(torch.int32)
    Q, kc, vc = (torch.randn(*s, generator=g).to(BF16) for s in ((1, Hq, d), (width, page, Hkv, d), (width, page, Hkv, d)))
    sel = torch.randperm(n, generator=g)[:k].sort().values
    idx = torch.full((1, k), -1, dtype=torch.int32)
    idx[0, :len(sel)] = sel.to(torch.int32)
    return Q, kc, vc, idx, table, sel


def attend(Q, kc, vc, idx, table, n, **kw):
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    O, lse = dsa.sparse_attn_decode_paged(Q.cuda(), kc.cuda(), vc.cuda(), idx.cuda(), table.cuda(), lens, **kw)
    return O[0].cpu(), lse[0].cpu()


def plain(Q, K, V, scale):
    """O [Hq, d] and lse [Hq] of one row in 64 bits, and the bound on a finite O (the paged attention's:
    weights to 2^-16, logits and exponentials 2e-4, the output's own rounding)."""
    G = Q.shape[0] // K.shape[1]
    K, V = (x.double().repeat_interleave(G, 1).transpose(0, 1) for x in (K, V))
    x = (K @ Q.double()[:, :, None])[:, :, 0] * scale
    m = x.amax(1, keepdim=True)
    p = torch.exp(x - m)
    total = p.sum(1, keepdim=True)
    O = ((p / total)[:, :, None] * V).sum(1)
    spread = ((p / total)[:, :, None] * (V - O[:, None]).abs()).sum(1)
    return O, (m + torch.log(total))[:, 0], (2.0 ** -16 + 2e-4) * spread + 2.0 ** -8 * O.abs() * 1.01 + 1e-6


def same_where_not_finite(got, want):
    """Infinities of the same sign and NaN in the same places; returns where both are finite."""
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan())
    inf = want.isinf()
    assert torch.equal(got.isinf(), inf) and torch.equal(got[inf], want[inf])
    return want.isfinite()


SHAPES = [(32, 4, 128), (8, 2, 64)]


@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
@pytest.mark.parametrize("n,k", [(1, 16), (20, 32), (700, 512), (3000, 2048)])
def test_infinity_in_a_selected_value(Hq, Hkv, d, n, k):
    """A weight times an infinity is that infinity; opposite ones, and NaN, give NaN; the other dims and
    KV heads stay finite."""
    page = 16
    Q, kc, vc, idx, table, sel = pages(Hq, Hkv, d, page, n, k, n + d)

    def put(s, head, dim, value):
        s = int(s)
        vc[int(table[0, s // page]), s % page, head, dim] = value

    put(sel[-1], 0, 3, INF)
    put(sel[0], 0, 4, -INF)
    put(sel[len(sel) // 2], 1, d - 1, -INF)
    if n > 1:
        put(sel[1], 1, 0, INF)
        put(sel[-2], 1, 0, INF)
        put(sel[1], 0, 7, INF)
        put(sel[-1], 0, 7, -INF)
        put(sel[2], 1, 9, NAN)
    O, lse = attend(Q, kc, vc, idx, table, n)
    at = table[0].long()[sel // page], sel % page
    want, wlse, bound = plain(Q[0], kc[at], vc[at], d ** -0.5)
    assert bool(want.isinf().any())
    fin = same_where_not_finite(O, want)
    assert bool(((O.double() - want).abs() <= bound)[fin].all())
    assert float((lse.double() - wlse).abs().max()) <= 5e-4


@pytest.mark.parametrize("Hq,Hkv,d", SHAPES)
@pytest.mark.parametrize("n,k", [(1, 16), (40, 48), (3000, 2048)])
@pytest.mark.parametrize("value", [NAN, INF])
def test_nan_reaches_lse(Hq, Hkv, d, n, k, value):
    """A NaN or an infinite logit makes the row's lse NaN: -inf says that nothing was selected."""
    page = 32
    Q, kc, vc, idx, table, sel = pages(Hq, Hkv, d, page, n, k, n + d + 1)
    Q = Q.abs() + 0.5  # an infinite key gives an infinite logit
    s, G = int(sel[len(sel) // 2]), Hq // Hkv
    kc[int(table[0, s // page]), s % page, 1] = value
    O, lse = attend(Q, kc, vc, idx, table, n)
    hit = torch.arange(Hq) // G == 1
    assert bool(lse[hit].isnan().all()) and bool(O[hit].isnan().all())
    at = table[0].long()[sel // page], sel % page
    want, wlse, bound = plain(Q[0], kc[at], vc[at], d ** -0.5)
    assert bool(((O.double() - want).abs() <= bound)[~hit].all())
    # logits of 128 products up to 60 in size: fp32 sums are off by 128 * 2^-24 * 60 = 4.6e-4
    assert float((lse.double() - wlse).abs()[~hit].max()) <= 1e-3
    # the masked kind does not count: the same value in a position that is not selected
    empty = torch.full_like(idx, -1)
    O, lse = attend(Q, kc, vc, empty, table, n)
    assert bool((O == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("H_I,d_I", [(64, 128), (32, 128), (16, 128), (8, 64), (4, 32)])
@pytest.mark.parametrize("page", [16, 256])
def test_indexer_scores_carry_nan_and_infinity(H_I, d_I, page):
    """A NaN in a key makes its score NaN and no other; one in the query, the whole row; an infinite
    product counts as it is where it is positive and as 0 where it is negative."""
    g = torch.Generator().manual_seed(H_I + page)
    lens = [300, 131, 1, 0, 77]
    pool = sum((n + page - 1) // page for n in lens) + 1
    table = ref.page_table(lens, page, pool, g)
    q = (torch.randint(0, 2, (5, H_I, d_I), generator=g) * 2 - 1).to(BF16)  # +-1: no product of 0 and infinity
    cache = torch.randint(-8, 9, (pool, page, d_I), generator=g).to(BF16)
    w = (0.5 ** torch.randint(1, 4, (5, H_I), generator=g)).to(BF16)

    def put(b, s, dim, value):
        cache[int(table[b, s // page]), s % page, dim] = value

    put(0, 0, 1, NAN), put(0, 127, 0, -NAN), put(0, 299, d_I - 1, NAN), put(1, 130, 5, NAN)
    put(0, 128, 2, INF), put(1, 7, 3, -INF), put(2, 0, 4, INF)
    q[4, 1, 2] = NAN
    unused = torch.ones(pool, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        s = torch.arange(n)
        unused[table[b].long()[s // page], s % page] = False
    cache[unused] = NAN  # behind the lengths and on pages of no sequence
    dev = [x.cuda() for x in (q, cache, w, table, torch.tensor(lens, dtype=torch.int32))]
    scores = dsa.index_paged(*dev, 300).cpu()
    for b, n in enumerate(lens):
        assert bool((scores[b, n:] == -INF).all())
        if n == 0:
            continue
        dots = torch.einsum("hd,sd->hs", q[b].double(), ref.f64(ref.cached(cache, table, b, n, page)))
        want = (w[b].double()[:, None] * torch.where(dots < 0, 0.0, dots)).sum(0)  # a NaN product stays
        fin = same_where_not_finite(scores[b, :n], want)
        assert torch.equal(scores[b, :n].double()[fin], want[fin]), b
    assert bool(scores[4, :77].isnan().all()) and int(scores[0, :300].isnan().sum()) == 3
    # through the decode: the sets of NaN scores are sets all the same, NaN first
    k = 16
    kc = torch.randn(pool, page, 2, 64, generator=g).to(BF16).cuda()
    Q = torch.randn(5, 8, 64, generator=g).to(BF16).cuda()
    idx, O, lse = dsa.decode_paged(dev[0], dev[2], Q, kc, kc, dev[1], dev[3], dev[4], 300, k)
    idx = idx.cpu()
    for b, n in enumerate(lens):
        sel = idx[b][idx[b] >= 0]
        assert len(sel) == min(k, n) == len(sel.unique()) and bool((sel < n).all())
    assert {0, 127, 299} <= set(idx[0].tolist()) and 130 in idx[1].tolist()
    assert bool(O.isfinite().all())
