"""Appending to a paged cache, the indexer scores and the attention over it, and the decode
pipelines that run them together, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import lightning_indexer_b200 as dsa
import paged_testutil as ref
from oracle import dsa_oracle as orc

pytestmark = pytest.mark.gpu

EPS = 1e-6
BF16 = torch.bfloat16


def randn(*shape, gen, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(BF16)


def weight(d, gen):
    return (1 + 0.3 * torch.randn(d, generator=gen)).to(BF16)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32)


# ------------------------------------------------------------------------------- append
@pytest.mark.parametrize("page,Hkv,d,d_I,rotary,irotary,inter,norm,given", [
    (16, 4, 128, 128, 128, 64, (False, False), True, False),
    (64, 2, 64, 32, 32, 32, (True, False), True, True),
    (1024, 1, 128, 64, 64, 64, (False, True), False, False),
    (32, 5, 64, 128, 16, 128, (True, True), True, True),
    (128, 3, 32, 128, 0, 0, (False, False), False, False),
])
def test_cache_append(page, Hkv, d, d_I, rotary, irotary, inter, norm, given):
    g = torch.Generator().manual_seed(page + d)
    # new tokens: 0, 1, a run over several pages, a whole new sequence, one that ends at a page's edge
    new = [0, 1, 37, 21, 16]
    lens = [9, 5, 60, 21, 2 * page]
    T = sum(new) + 5  # rows behind the last sequence
    cu = i32([2] + (2 + np.cumsum(new)).tolist())  # and two before the first
    pool = sum((n + page - 1) // page for n in lens) + 2
    table = ref.page_table(lens, page, pool, g)
    K, V, I = randn(T, Hkv, d, gen=g), randn(T, Hkv, d, gen=g), randn(T, d_I, gen=g)
    gk, gi = (weight(d, g), weight(d_I, g)) if norm else (None, None)
    freq, ifreq = ref.frequencies(rotary) if rotary else None, ref.frequencies(irotary, 5e5) if irotary else None
    positions = torch.randint(0, 500_000, (T,), generator=g, dtype=torch.int32) if given else None
    # one allocation holds both caches by turns: the page strides are larger than a page
    kv = randn(pool, 2, page, Hkv, d, gen=g).cuda()
    ic = randn(pool, page, d_I, gen=g).cuda()
    kv0, ic0 = kv.cpu(), ic.cpu()
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    dsa.cache_append(K.cuda(), V.cuda(), I.cuda(), kv[:, 0], kv[:, 1], ic, table.cuda(), cu.cuda(), i32(lens).cuda(), k_weight=dev(gk),
                     k_idx_weight=dev(gi), inv_freq=dev(freq), idx_inv_freq=dev(ifreq), positions=dev(positions), interleaved=inter[0],
                     idx_interleaved=inter[1], eps=EPS)
    kv, ic = kv.cpu(), ic.cpu()
    written = torch.zeros(pool, page, dtype=torch.bool)
    for b, n in enumerate(new):
        for i in range(n):
            t, p = int(cu[b]) + i, lens[b] - n + i
            at = int(table[b, p // page]), p % page
            written[at] = True
            rot = positions[t:t + 1] if given else torch.tensor([p])
            assert torch.equal(kv[at[0], 1, at[1]], V[t])
            for got, x, w, f, il in ((kv[at[0], 0, at[1]], K[t], gk, freq, inter[0]), (ic[at][None], I[t][None], gi, ifreq, inter[1])):
                x, w = ref.f64(x)[None], None if w is None else ref.f64(w)
                want = ref.norm_rope(x, w, EPS, rot, f, il)
                assert bool(((ref.f64(got)[None] - want).abs() <= ref.norm_rope_tolerance(x, w, EPS, want)).all())
    assert int(written.sum()) == sum(new)
    assert torch.equal(kv.transpose(1, 2)[~written], kv0.transpose(1, 2)[~written]) and torch.equal(ic[~written], ic0[~written])


def test_cache_append_drops_tokens_without_a_page():
    g = torch.Generator().manual_seed(1)
    page, pool, Hkv, d, d_I = 16, 6, 2, 64, 64
    # sequence 0: more new tokens than its length; 1: a page outside the pool and one that is -1;
    # 2: past the table's width; 3: a negative length
    new, lens = [8, 40, 20, 3], [5, 40, 70, -7]
    table = i32([[0, -1, -1], [6, 1, -1], [2, 3, 4], [5, 5, 5]])
    T, cu = sum(new), i32([0] + np.cumsum(new).tolist())
    K, V, I = randn(T, Hkv, d, gen=g), randn(T, Hkv, d, gen=g), randn(T, d_I, gen=g)
    kc, vc, ic = (torch.zeros(pool, page, *s, dtype=BF16, device="cuda") for s in ((Hkv, d), (Hkv, d), (d_I,)))
    dsa.cache_append(K.cuda(), V.cuda(), I.cuda(), kc, vc, ic, table.cuda(), cu.cuda(), i32(lens).cuda())
    want = torch.zeros(pool, page, Hkv, d, dtype=BF16)
    for b in range(4):
        for i in range(new[b]):
            p = lens[b] - new[b] + i
            if 0 <= p < 48 and 0 <= int(table[b, p // page]) < pool:
                want[int(table[b, p // page]), p % page] = V[int(cu[b]) + i]
    assert torch.equal(vc.cpu(), want) and int((want != 0).any(-1).any(-1).sum()) == 5 + 16
    # without indexer keys
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    dsa.cache_append(K.cuda(), V.cuda(), None, kc2, vc2, None, table.cuda(), cu.cuda(), i32(lens).cuda())
    assert torch.equal(kc2, kc) and torch.equal(vc2, vc)


def test_cache_append_many_tokens():
    """A prefill's worth of rows (several row groups per warp) equals norm_rope's rows, bit for bit."""
    g = torch.Generator().manual_seed(2)
    page, Hkv, d, d_I, new = 64, 4, 128, 128, [3001, 5200]
    T, cu = sum(new), i32([0, 3001, 8201])
    pool = sum((n + page - 1) // page for n in new)
    table = ref.page_table(new, page, pool, g)
    K, V, I = randn(T, Hkv, d, gen=g).cuda(), randn(T, Hkv, d, gen=g).cuda(), randn(T, d_I, gen=g).cuda()
    w, wi, f = weight(d, g).cuda(), weight(d_I, g).cuda(), ref.frequencies(128).cuda()
    kc, vc = (torch.zeros(pool, page, Hkv, d, dtype=BF16, device="cuda") for _ in range(2))
    ic = torch.zeros(pool, page, d_I, dtype=BF16, device="cuda")
    dsa.cache_append(K, V, I, kc, vc, ic, table.cuda(), cu.cuda(), i32(new).cuda(), k_weight=w, k_idx_weight=wi, inv_freq=f, idx_inv_freq=f)
    Kr, Ir = dsa.norm_rope(K, None, w, None, f, cu_seqlens_q=cu.cuda())[0], dsa.norm_rope(I[:, None], None, wi, None, f, cu_seqlens_q=cu.cuda())[0]
    for b in range(2):
        lo, hi = int(cu[b]), int(cu[b + 1])
        for cache, rows in ((kc, Kr), (vc, V), (ic, Ir[:, 0])):
            assert torch.equal(ref.cached(cache.cpu(), table, b, new[b], page), rows[lo:hi].cpu())


# ------------------------------------------------------------------------- indexer scores
LENS = [1000, 0, 1, 127, 128, 129, 15, 16, 17, 641, 0, 300]


@pytest.mark.parametrize("H_I,d_I", [(64, 128), (32, 128), (16, 128), (8, 64), (4, 32)])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("integer", [True, False])
def test_index_paged(H_I, d_I, page, integer):
    g = torch.Generator().manual_seed(H_I + page)
    lens, B = LENS, len(LENS)
    pool = sum((n + page - 1) // page for n in lens) + 1
    table = ref.page_table(lens, page, pool, g)
    if integer:  # exact in fp32 in any order: products of integers up to 8, weights 1/2, 1/4, 1/8
        q = torch.randint(-8, 9, (B, H_I, d_I), generator=g).to(BF16)
        cache = torch.randint(-8, 9, (pool, page, d_I), generator=g).to(BF16)
        w = (0.5 ** torch.randint(1, 4, (B, H_I), generator=g)).to(BF16)
    else:
        q, cache = randn(B, H_I, d_I, gen=g), randn(pool, page, d_I, gen=g)
        w = torch.softmax(torch.randn(B, H_I, generator=g), 1).to(BF16)
    ld = 1004
    scores = torch.full((B, ld), 123.0, device="cuda")
    strided = torch.zeros(pool, 2, page, d_I, dtype=BF16, device="cuda")
    strided[:, 0] = cache.cuda()
    dsa.index_paged(q.cuda(), strided[:, 0], w.cuda(), table.cuda(), i32(lens).cuda(), 1000, scores=scores)
    scores = scores.cpu()
    for b, n in enumerate(lens):
        assert bool((scores[b, n:] == 123.0).all())
        if n == 0:
            continue
        dots = ref.f64(q[b]) @ ref.f64(ref.cached(cache, table, b, n, page)).T
        want = ref.f64(w[b]) @ dots.clamp(min=0)
        # fp32 sums of d_I products and H_I heads: (128 + 64) 2^-24 = 1.1e-5 of the row's scale
        tol = 0.0 if integer else 2e-5 * float(want.abs().max()) + 1e-6
        assert float((ref.f64(scores[b, :n]) - want).abs().max()) <= tol, (b, n)


def test_index_paged_many_sequences_and_bad_pages():
    g = torch.Generator().manual_seed(5)
    B, H_I, d_I, page = 421, 32, 128, 32  # more sequences than threads of a block
    lens = torch.randint(0, 200, (B,), generator=g).tolist()
    lens[7], lens[8], lens[420] = 100000, -3, 199  # cut at max_seqlen_k; counts as empty
    cut = [min(max(n, 0), 200) for n in lens]
    pool = 40  # pages are shared by many sequences
    table = torch.randint(0, pool, (B, 7), generator=g, dtype=torch.int32)
    bad = torch.rand(B, 7, generator=g) < 0.1
    table[bad] = torch.where(torch.rand(int(bad.sum()), generator=g) < 0.5, -1, pool).to(torch.int32)
    q = torch.randint(-8, 9, (B, H_I, d_I), generator=g).to(BF16)
    cache = torch.randint(-8, 9, (pool, page, d_I), generator=g).to(BF16)
    w = (0.5 ** torch.randint(1, 4, (B, H_I), generator=g)).to(BF16)
    scores = dsa.index_paged(q.cuda(), cache.cuda(), w.cuda(), table.cuda(), i32(lens).cuda(), 200).cpu()
    assert scores.shape == (B, 200)
    for b, n in enumerate(cut):
        s = torch.arange(n)
        pages = table[b].long()[s // page]
        there = (pages >= 0) & (pages < pool)
        k = ref.f64(cache[pages.clamp(0, pool - 1), s % page])
        want = ref.f64(w[b]) @ (ref.f64(q[b]) @ k.T).clamp(min=0)
        want[~there] = float("-inf")
        assert torch.equal(ref.f64(scores[b, :n]), want), b
        assert bool((scores[b, n:] == float("-inf")).all())


def test_index_paged_length_past_the_table():
    """A length past max_pages * page_size is cut there; the score columns behind stay as they were."""
    g = torch.Generator().manual_seed(6)
    page, lens = 16, [300, 33, 48]
    q, cache, w = integer_pool(3, 16, 128, 9, page, g)
    table = torch.randperm(9, generator=g).view(3, 3).to(torch.int32)
    scores = torch.full((3, 304), 5.0, device="cuda")
    dsa.index_paged(q.cuda(), cache.cuda(), w.cuda(), table.cuda(), i32(lens).cuda(), 300, scores=scores)
    for b, n in enumerate([48, 33, 48]):
        want = ref.f64(w[b]) @ (ref.f64(q[b]) @ ref.f64(ref.cached(cache, table, b, n, page)).T).clamp(min=0)
        assert torch.equal(ref.f64(scores[b, :n]), want) and bool((scores[b, n:] == 5.0).all())


def test_index_paged_no_keys():
    q, w = torch.zeros(3, 64, 128, dtype=BF16, device="cuda"), torch.zeros(3, 64, dtype=BF16, device="cuda")
    cache = torch.zeros(1, 16, 128, dtype=BF16, device="cuda")
    scores = dsa.index_paged(q, cache, w, torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), 0)
    assert bool((scores == float("-inf")).all())


# ------------------------------------------------------------------------------ attention
def attention(Q, K, V, scale):
    """(O, lse, bound on |O - exact|) of one row: Q [Hq, d], K, V [n, Hkv, d] in 64 bits.

    The bound: the weights are held as two bf16, what the first rounds off in the second, so each is
    off by at most 2^-16 of itself; the fp32 logits (sums of 128 products) and exponentials move it
    by less than 2e-4; O moves by that times sum p |V - O|, and its own rounding is 2^-8 |O|."""
    Hq, Hkv = Q.shape[0], K.shape[1]
    if K.shape[0] == 0:
        return torch.zeros_like(Q), torch.full((Hq,), -math.inf, dtype=torch.float64), torch.zeros_like(Q)
    K, V = (x.repeat_interleave(Hq // Hkv, 1).transpose(0, 1) for x in (K, V))  # [Hq, n, d]
    x = (K @ Q[:, :, None])[:, :, 0] * scale
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])[:, None]
    O = (p @ V)[:, 0]
    spread = (p @ (V - O[:, None]).abs())[:, 0]
    return O, lse, (2.0 ** -16 + 2e-4) * spread + 2.0 ** -8 * O.abs() * 1.01 + 1e-6


LSE_ATOL = 5e-4  # a logit of 128 products (5e-5), ex2 (2^-22) and fp32 sums of up to 4096 terms (2.4e-4)


def make_attention_case(Hq, Hkv, d, k, page, lens, seed):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pool = sum((n + page - 1) // page for n in lens) + 2
    table = ref.page_table(lens, page, pool, g)
    Q, kc, vc = randn(B, Hq, d, gen=g), randn(pool, page, Hkv, d, gen=g), randn(pool, page, Hkv, d, gen=g)
    idx = torch.full((B, k), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        sel = torch.randperm(n, generator=g)[:k].sort().values
        idx[b, :len(sel)] = sel.to(torch.int32)
    return Q, kc, vc, idx, table, g


@pytest.mark.parametrize("Hq,Hkv,d", [(32, 4, 128), (20, 5, 64), (8, 2, 64), (8, 1, 128), (16, 4, 128)])
@pytest.mark.parametrize("k,page", [(16, 16), (48, 64), (208, 32), (2048, 128)])
def test_attention_paged(Hq, Hkv, d, k, page):
    lens = [700, 0, 1, 15, 2500, 16, 33]
    Q, kc, vc, idx, table, _ = make_attention_case(Hq, Hkv, d, k, page, lens, k + Hq)
    O, lse = dsa.sparse_attn_decode_paged(Q.cuda(), kc.cuda(), vc.cuda(), idx.cuda(), table.cuda(), i32(lens).cuda())
    for b, n in enumerate(lens):
        s = idx[b][idx[b] >= 0].long()
        at = table[b].long()[s // page], s % page
        want, wlse, bound = attention(ref.f64(Q[b]), ref.f64(kc[at]), ref.f64(vc[at]), d ** -0.5)
        assert bool(((ref.f64(O[b]) - want).abs() <= bound).all()), (b, n)
        assert torch.equal(torch.isinf(wlse), torch.isinf(lse[b].cpu()))
        assert n == 0 or float((ref.f64(lse[b]) - wlse).abs().max()) <= LSE_ATOL
    # again: the same bits; one row alone, without the lse, is split differently and meets the same bound
    again = dsa.sparse_attn_decode_paged(Q.cuda(), kc.cuda(), vc.cuda(), idx.cuda(), table.cuda(), i32(lens).cuda())
    assert torch.equal(again[0], O) and torch.equal(again[1], lse)
    one = torch.empty(1, Hq, d, dtype=BF16, device="cuda")
    dsa.sparse_attn_decode_paged(Q[4:5].cuda(), kc.cuda(), vc.cuda(), idx[4:5].cuda(), table[4:5].cuda(), i32(lens[4:5]).cuda(), out=(one, None))
    s = idx[4][idx[4] >= 0].long()
    at = table[4].long()[s // page], s % page
    want, _, bound = attention(ref.f64(Q[4]), ref.f64(kc[at]), ref.f64(vc[at]), d ** -0.5)
    assert bool(((ref.f64(one[0]) - want).abs() <= bound).all())


@pytest.mark.parametrize("B", [9, 36, 150])
def test_attention_paged_batches(B):
    """Batches on both sides of the split rule, every row against its bound."""
    page, d, k = 32, 64, 512
    lens = [(97 * b) % 1500 for b in range(B)]
    Q, kc, vc, idx, table, _ = make_attention_case(8, 2, d, k, page, lens, B)
    O, lse = dsa.sparse_attn_decode_paged(Q.cuda(), kc.cuda(), vc.cuda(), idx.cuda(), table.cuda(), i32(lens).cuda())
    for b, n in enumerate(lens):
        s = idx[b][idx[b] >= 0].long()
        at = table[b].long()[s // page], s % page
        want, wlse, bound = attention(ref.f64(Q[b]), ref.f64(kc[at]), ref.f64(vc[at]), d ** -0.5)
        assert bool(((ref.f64(O[b]) - want).abs() <= bound).all()), (b, n)
        assert n == 0 or float((ref.f64(lse[b]) - wlse).abs().max()) <= LSE_ATOL


def test_attention_ignores_what_is_not_there():
    """Entries outside the length, on pages outside the pool or past the table do not count, whatever
    the cache holds there; unused rows of the pool may hold NaN."""
    page, lens, k, d = 16, [40, 64, 30, 100], 64, 128
    Q, kc, vc, idx, table, g = make_attention_case(32, 4, d, k, page, lens, 3)
    pool = kc.shape[0]
    idx[0, 3], idx[0, 5], idx[0, 7] = 40, 2 ** 31 - 1, -2 ** 31
    table[1, 1], table[1, 3] = pool, -5
    table[2] = -1  # nothing there at all
    table = table[:, :4].contiguous()  # sequence 3 reaches past the table
    used = torch.zeros(pool, page, dtype=torch.bool)
    rows = []
    for b, n in enumerate(lens):
        s = idx[b].long()
        s = s[(s >= 0) & (s < n) & (s < 64)]
        pg = table[b].long()[s // page]
        s, pg = s[(pg >= 0) & (pg < pool)], pg[(pg >= 0) & (pg < pool)]
        used[pg, s % page] = True
        rows.append((pg, s % page))
    kc[~used], vc[~used] = float("nan"), float("inf")
    O, lse = dsa.sparse_attn_decode_paged(Q.cuda(), kc.cuda(), vc.cuda(), idx.cuda(), table.cuda(), i32(lens).cuda())
    for b, at in enumerate(rows):
        want, wlse, bound = attention(ref.f64(Q[b]), ref.f64(kc[at]), ref.f64(vc[at]), d ** -0.5)
        assert bool(((ref.f64(O[b]) - want).abs() <= bound).all()), b
        assert bool((lse[b].cpu() == -math.inf).all()) if len(at[0]) == 0 else float((ref.f64(lse[b]) - wlse).abs().max()) <= LSE_ATOL
    assert bool((O[2] == 0).all())


def test_attention_paged_rising_logits_scale_and_duplicates():
    """Logits that rise past the held maximum chunk by chunk; a given scale; a position named twice counts twice."""
    page, n, k, d = 32, 512, 512, 64
    Q, kc, vc, idx, table, g = make_attention_case(8, 2, d, k, page, [n], 4)
    Q[:] = 1.0
    s = torch.arange(n)
    kc[table[0].long()[s // page], s % page] = (s[:, None, None] * (60.0 / n) * torch.ones(1, 2, d) / d).to(BF16)
    idx[0, 9] = idx[0, 400] = 500
    O, lse = dsa.sparse_attn_decode_paged(Q.cuda(), kc.cuda(), vc.cuda(), idx.cuda(), table.cuda(), i32([n]).cuda(), scale=1.25)
    at = table[0].long()[idx[0].long() // page], idx[0].long() % page
    want, wlse, bound = attention(ref.f64(Q[0]), ref.f64(kc[at]), ref.f64(vc[at]), 1.25)
    assert bool(((ref.f64(O[0]) - want).abs() <= bound).all())
    # logits up to 75: their fp32 sums of 64 products are off by 64 * 2^-24 * 75 = 3e-4
    assert float((ref.f64(lse[0]) - wlse).abs().max()) <= LSE_ATOL + 3e-4


def test_attention_strided_pages():
    page, lens, k, d, Hkv = 16, [333, 90], 128, 128, 4
    Q, kc, vc, idx, table, _ = make_attention_case(32, Hkv, d, k, page, lens, 6)
    kv = torch.stack([kc, vc], 1).cuda()  # [pool, 2, page, Hkv, d]
    a = dsa.sparse_attn_decode_paged(Q.cuda(), kv[:, 0], kv[:, 1], idx.cuda(), table.cuda(), i32(lens).cuda())
    b = dsa.sparse_attn_decode_paged(Q.cuda(), kc.cuda(), vc.cuda(), idx.cuda(), table.cuda(), i32(lens).cuda())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("Hq,Hkv,d,k", [(32, 4, 128, 128), (16, 4, 64, 4096), (8, 1, 128, 1040)])
def test_attention_page_strides_differ(Hq, Hkv, d, k):
    """Key and value pages spaced apart differently, and the largest sets."""
    page, lens = 32, [4500, 90]
    Q, kc, vc, idx, table, _ = make_attention_case(Hq, Hkv, d, k, page, lens, 8)
    n = page * Hkv * d
    wide = torch.full((kc.shape[0], n + 264), float("nan"), dtype=BF16, device="cuda")
    kw = wide[:, 8:8 + n].unflatten(1, (page, Hkv, d))
    kw.copy_(kc)
    O, lse = dsa.sparse_attn_decode_paged(Q.cuda(), kw, vc.cuda(), idx.cuda(), table.cuda(), i32(lens).cuda())
    for b in range(2):
        s = idx[b][idx[b] >= 0].long()
        at = table[b].long()[s // page], s % page
        want, wlse, bound = attention(ref.f64(Q[b]), ref.f64(kc[at]), ref.f64(vc[at]), d ** -0.5)
        assert bool(((ref.f64(O[b]) - want).abs() <= bound).all())
        assert float((ref.f64(lse[b]) - wlse).abs().max()) <= LSE_ATOL


def test_far_offsets():
    """Elements past 2^31 in a cache whose pages lie far apart."""
    page, d, Hkv, d_I = 16, 64, 2, 64
    far = torch.zeros(4, 1 << 29, dtype=BF16, device="cuda")  # 4 GiB; page stride 2^29 elements
    kc, vc = (far[:, o:o + page * Hkv * d].unflatten(1, (page, Hkv, d)) for o in (0, 4096))
    ic = far[:, 8192:8192 + page * d_I].unflatten(1, (page, d_I))
    g = torch.Generator().manual_seed(7)
    T = 40
    K, V, I = randn(T, Hkv, d, gen=g), randn(T, Hkv, d, gen=g), torch.randint(-8, 9, (T, d_I), generator=g).to(BF16)
    table, lens, cu = i32([[3, 0, 2]]).cuda(), i32([T]).cuda(), i32([0, T]).cuda()
    dsa.cache_append(K.cuda(), V.cuda(), I.cuda(), kc, vc, ic, table, cu, lens)
    for cache, rows in ((kc, K), (vc, V), (ic, I)):
        assert torch.equal(torch.cat([cache[3], cache[0], cache[2][:8]]).cpu(), rows)
    Q = randn(1, 8, d, gen=g)
    idx = i32([list(range(T)) + [-1] * 8])
    O, _ = dsa.sparse_attn_decode_paged(Q.cuda(), kc, vc, idx.cuda(), table, lens)
    want, _, bound = attention(ref.f64(Q[0]), ref.f64(K), ref.f64(V), d ** -0.5)
    assert bool(((ref.f64(O[0]) - want).abs() <= bound).all())
    q = torch.randint(-8, 9, (1, 8, d_I), generator=g).to(BF16)
    w = (0.5 ** torch.randint(1, 4, (1, 8), generator=g)).to(BF16)
    scores = dsa.index_paged(q.cuda(), ic, w.cuda(), table, lens, T)
    assert torch.equal(ref.f64(scores[0]), ref.f64(w[0]) @ (ref.f64(q[0]) @ ref.f64(I).T).clamp(min=0))


# --------------------------------------------------------------------------- all together
def integer_pool(B, H_I, d_I, pool, page, g):
    q = torch.randint(-8, 9, (B, H_I, d_I), generator=g).to(BF16)
    cache = torch.randint(-8, 9, (pool, page, d_I), generator=g).to(BF16)
    w = (0.5 ** torch.randint(1, 4, (B, H_I), generator=g)).to(BF16)
    return q, cache, w


@pytest.mark.parametrize("lens,page,k,H_I,d_I", [([3000, 0, 17, 2048, 5000], 64, 256, 64, 128), ([40000, 70001], 128, 2048, 64, 128),
                                                 ([900], 16, 128, 4, 32)])
def test_decode_paged_equals_contiguous_decode(lens, page, k, H_I, d_I):
    """The same sets as the contiguous decode and the oracle (exact scores), attention within its bound."""
    Hq, Hkv, d, B = (32, 4, 128, len(lens)) if d_I == 128 else (8, 2, 64, len(lens))
    Q, kc, vc, _, table, g = make_attention_case(Hq, Hkv, d, 16, page, lens, 11)
    q, ic, w = integer_pool(B, H_I, d_I, kc.shape[0], page, g)
    args = [x.cuda() for x in (q, w, Q, kc, vc, ic, table)] + [i32(lens).cuda()]
    idx, O, lse = dsa.decode_paged(*args, max(lens), k)
    Kp, Vp, Ip = (torch.cat([ref.cached(x, table, b, n, page) for b, n in enumerate(lens)]) for x in (kc, vc, ic))
    cu = i32(np.concatenate([[0], np.cumsum(lens)]))
    want = dsa.decode(q.cuda(), Ip.cuda(), w.cuda(), Q.cuda(), Kp.cuda(), Vp.cuda(), cu.cuda(), max(lens), k)
    assert torch.equal(idx, want[0])
    for b, n in enumerate(lens):
        dots = (ref.f64(q[b]) @ ref.f64(ref.cached(ic, table, b, n, page)).T).clamp(min=0)
        sel = orc.topk_row((ref.f64(w[b]) @ dots).numpy(), k)
        assert np.array_equal(idx[b].cpu().numpy()[:len(sel)], sel)
        s = idx[b][idx[b] >= 0].long().cpu()
        at = table[b].long()[s // page], s % page
        o, l, bound = attention(ref.f64(Q[b]), ref.f64(kc[at]), ref.f64(vc[at]), d ** -0.5)
        assert bool(((ref.f64(O[b]) - o).abs() <= bound).all()), b
        assert n == 0 or float((ref.f64(lse[b]) - l).abs().max()) <= LSE_ATOL
    assert dsa.device_status() == (0, 0)


@pytest.mark.parametrize("norm,given", [(True, False), (False, True)])
def test_decode_step_is_its_parts(norm, given):
    """One step from the projections equals norm_rope, cache_append and decode_paged, bit for bit; then
    a second step on the grown cache."""
    g = torch.Generator().manual_seed(13)
    page, Hq, Hkv, d, H_I, d_I, k = 32, 32, 4, 128, 64, 128, 64
    lens = [101, 1, 64, 33, 0, 250]
    B, width = len(lens), 9
    pool = B * width
    table = torch.randperm(pool, generator=g).view(B, width).to(torch.int32).cuda()
    kc, vc = randn(pool, page, Hkv, d, gen=g).cuda(), randn(pool, page, Hkv, d, gen=g).cuda()
    ic = randn(pool, page, d_I, gen=g).cuda()
    gq, gk, gqi, gki = (weight(n, g).cuda() if norm else None for n in (d, d, d_I, d_I))
    f, fi = ref.frequencies(128).cuda(), ref.frequencies(64).cuda()
    caches = [x.clone() for x in (kc, vc, ic)]
    ws = torch.full((dsa.decode_step_paged_workspace_bytes(B, 288, Hq, d, H_I, d_I),), 255, dtype=torch.uint8, device="cuda")
    for step in range(2):
        x = randn(B, (Hq + 2 * Hkv) * d, gen=g).cuda()
        Q, K, V = (x[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        y = randn(B, (H_I + 1) * d_I, gen=g).cuda()
        qi, ki = y[:, :H_I * d_I].unflatten(1, (H_I, d_I)), y[:, H_I * d_I:]
        w = torch.softmax(torch.randn(B, H_I, generator=g), 1).to(BF16).cuda()
        n = i32([m + step if m else 0 for m in lens]).cuda()
        pos = torch.randint(0, 9999, (B,), generator=g, dtype=torch.int32).cuda() if given else None
        got = dsa.decode_step_paged(qi, w, Q, K, V, ki, kc, vc, ic, table, n, 288, k, gq, gk, gqi, gki, f, fi, positions=pos,
                                    idx_interleaved=True, workspace=ws)
        cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        Qr, _ = dsa.norm_rope(Q, None, gq, None, f, positions=pos, cu_seqlens_q=cu, seqlens_k=n)
        qir, _ = dsa.norm_rope(qi, None, gqi, None, fi, positions=pos, cu_seqlens_q=cu, seqlens_k=n, interleaved=True)
        dsa.cache_append(K, V, ki, *caches, table, cu, n, gk, gki, f, fi, pos, idx_interleaved=True)
        assert all(torch.equal(a, b) for a, b in zip((kc, vc, ic), caches))
        want = dsa.decode_paged(qir, w, Qr, *caches, table, n, 288, k)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert bool((got[0][4] == -1).all()) and bool((got[1][4] == 0).all()) and bool((got[2][4] == -math.inf).all())


def test_prefill_then_decode_equals_one_longer_prefill():
    """A prompt through norm_rope, prefill and cache_append, then one decode step: the step's output is
    the last row of a prefill that is one token longer."""
    g = torch.Generator().manual_seed(17)
    page, Hq, Hkv, d, H_I, d_I, n, k = 64, 32, 4, 128, 64, 128, 600, 1024  # k past the length: attention is dense
    Q, K, V = randn(n, Hq, d, gen=g).cuda(), randn(n, Hkv, d, gen=g).cuda(), randn(n, Hkv, d, gen=g).cuda()
    qi, ki = randn(n, H_I, d_I, gen=g).cuda(), randn(n, d_I, gen=g).cuda()
    w = torch.softmax(torch.randn(n, H_I, generator=g), 1).to(BF16).cuda()
    gq, gk, f, fi = weight(d, g).cuda(), weight(d, g).cuda(), ref.frequencies(d).cuda(), ref.frequencies(64).cuda()
    cu = i32([0, n]).cuda()
    Qr, Kr = dsa.norm_rope(Q, K, gq, gk, f, cu_seqlens_q=cu)
    qir, kir = dsa.norm_rope(qi, ki[:, None], None, None, fi, cu_seqlens_q=cu)
    idx, O, lse = dsa.prefill(qir, kir[:, 0].contiguous(), w, Qr, Kr, V, cu, cu, n, n, k)
    pool = (n + page - 1) // page
    table = torch.randperm(pool, generator=g)[None].to(torch.int32).cuda()
    kc, vc = (torch.zeros(pool, page, Hkv, d, dtype=BF16, device="cuda") for _ in range(2))
    ic = torch.zeros(pool, page, d_I, dtype=BF16, device="cuda")
    m = n - 1
    dsa.cache_append(K[:m], V[:m], ki[:m], kc, vc, ic, table, i32([0, m]).cuda(), i32([m]).cuda(), gk, None, f, fi)
    got = dsa.decode_step_paged(qi[m:], w[m:], Q[m:], K[m:], V[m:], ki[m:], kc, vc, ic, table, i32([n]).cuda(), n, k, gq, gk, None, None, f, fi)
    assert torch.equal(got[0][0], idx[m])
    assert torch.equal(ref.cached(kc.cpu(), table.cpu(), 0, n, page), Kr.cpu())
    want, wlse, bound = attention(ref.f64(Qr[m]), ref.f64(Kr), ref.f64(V), d ** -0.5)
    assert bool(((ref.f64(got[1][0]) - want).abs() <= bound).all())
    # the prefill rounds its weights to bf16, 2^-8 of sum p |V - O| <= 2 max |V| more than the step's bound
    assert bool(((ref.f64(O[m]) - ref.f64(got[1][0])).abs() <= 2 * bound + 2.0 ** -7 * ref.f64(V).abs().max()).all())
    assert float((ref.f64(got[2][0]) - ref.f64(lse[m])).abs().max()) <= 2 * LSE_ATOL


def test_decode_step_graph_two_streams():
    """A captured step replayed on changing inputs and lengths, and steps on two streams at once, each
    with its own workspace."""
    g = torch.Generator().manual_seed(19)
    page, Hq, Hkv, d, H_I, d_I, k, B, width = 16, 8, 2, 64, 8, 64, 32, 3, 8
    pool = B * width
    table = torch.randperm(pool, generator=g).view(B, width).to(torch.int32).cuda()

    def fresh(seed):
        h = torch.Generator().manual_seed(seed)
        return [randn(pool, page, Hkv, d, gen=h).cuda(), randn(pool, page, Hkv, d, gen=h).cuda(), randn(pool, page, d_I, gen=h).cuda()]

    def inputs(seed):
        h = torch.Generator().manual_seed(seed)
        w = torch.softmax(torch.randn(B, H_I, generator=h), 1).to(BF16)
        return [x.cuda() for x in (randn(B, H_I, d_I, gen=h), w, randn(B, Hq, d, gen=h), randn(B, Hkv, d, gen=h), randn(B, Hkv, d, gen=h),
                                   randn(B, d_I, gen=h), i32([50 + seed, 1 + seed, 128 - seed]))]

    f = ref.frequencies(64).cuda()

    def step(x, c, **kw):
        return dsa.decode_step_paged(*x[:6], *c, table, x[6], width * page, k, inv_freq=f, idx_inv_freq=f, **kw)

    cap, caches = inputs(0), fresh(1)
    step(cap, caches)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cap, caches)
    mirror = [c.clone() for c in caches]
    for seed in (1, 2, 3):
        x = inputs(seed)
        for a, b in zip(cap, x):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want = step(x, mirror)
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and all(torch.equal(a, b) for a, b in zip(caches, mirror))
    xs, cs = [inputs(5), inputs(6)], [fresh(5), fresh(6)]
    wants = [step(x, [t.clone() for t in c]) for x, c in zip(xs, cs)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s, x, c in zip(streams, xs, cs):
        with torch.cuda.stream(s):
            outs.append([step(x, c) for _ in range(6)])
    torch.cuda.synchronize()
    for runs, want in zip(outs, wants):
        assert all(torch.equal(a, b) for r in runs for a, b in zip(r, want))
    assert dsa.device_status() == (0, 0)


def test_dependent_steps_back_to_back():
    """Thirty decode steps, each appending to the cache that the next one reads and feeding it its
    output, give what they give with the device waited for after every call."""
    g = torch.Generator().manual_seed(29)
    page, Hq, Hkv, d, H_I, d_I, k, B, width = 16, 32, 4, 128, 64, 128, 64, 5, 16
    pool = B * width
    table = torch.randperm(pool, generator=g).view(B, width).to(torch.int32).cuda()
    start = [randn(pool, page, Hkv, d, gen=g), randn(pool, page, Hkv, d, gen=g), randn(pool, page, d_I, gen=g)]
    x0, f = randn(B, Hq, d, gen=g).cuda(), ref.frequencies(128).cuda()
    w = torch.softmax(torch.randn(B, H_I, generator=g), 1).to(BF16).cuda()
    lens = [i32([b * 37 + i + 1 for b in range(B)]).cuda() for i in range(30)]

    def run(wait):
        caches, x, out = [c.cuda() for c in start], x0, []
        for n in lens:
            K, qi = x[:, :Hkv].contiguous(), x.repeat(1, 2, 1)
            got = dsa.decode_step_paged(qi, w, x, K, K, x[:, 0], *caches, table, n, width * page, k, inv_freq=f, idx_inv_freq=f)
            if wait:
                torch.cuda.synchronize()
            x, _ = dsa.norm_rope(got[1], None, torch.ones(d, dtype=BF16, device="cuda"))
            if wait:
                torch.cuda.synchronize()
            out += [got[0], x]
        return out + caches

    assert all(torch.equal(a, b) for a, b in zip(run(False), run(True)))


def test_capture_with_a_second_stream():
    """A captured region in which a call's inputs come from another stream, and the call's outputs go
    back to it, replays as it ran."""
    g = torch.Generator().manual_seed(23)
    page, Hq, Hkv, d, k, lens = 16, 8, 2, 64, 64, [200, 77, 150]
    Q, kc, vc, idx, table, _ = make_attention_case(Hq, Hkv, d, k, page, lens, 23)
    x, w, f = randn(3, Hq, d, gen=g).cuda(), weight(d, g).cuda(), ref.frequencies(d).cuda()
    kc, vc, idx, table, n = kc.cuda(), vc.cuda(), idx.cuda(), table.cuda(), i32(lens).cuda()
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            q, _ = dsa.norm_rope(x * 2, None, w, None, f, cu_seqlens_q=cu, seqlens_k=n)
        main.wait_stream(side)
        O, lse = dsa.sparse_attn_decode_paged(q, kc, vc, idx, table, n)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            y, _ = dsa.norm_rope(O, None, w)
        main.wait_stream(side)
        return q, O, lse, y

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for seed in (1, 2, 3):
        x.copy_(randn(3, Hq, d, gen=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_checks_sizes():
    """Sizes that would make a kernel read past a tensor are refused before anything is enqueued."""
    z = lambda *s, t=BF16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    i = lambda *s: z(*s, t=torch.int32)  # noqa: E731
    Q, w128, f = z(4, 8, 128), z(128), torch.zeros(64, dtype=torch.float64, device="cuda")
    bad = [lambda: dsa.norm_rope(Q, z(3, 2, 128)), lambda: dsa.norm_rope(Q, None, z(64)), lambda: dsa.norm_rope(Q, None, w128.float()),
           lambda: dsa.norm_rope(Q, None, None, None, f.float()), lambda: dsa.norm_rope(Q, None, None, None, f, positions=i(3)),
           lambda: dsa.norm_rope(Q, None, None, None, f, positions=z(4, t=torch.int64)), lambda: dsa.norm_rope(Q, seqlens_k=i(4), cu_seqlens_q=i(4)),
           lambda: dsa.norm_rope(Q[:, ::2]), lambda: dsa.norm_rope(Q[..., ::2]), lambda: dsa.norm_rope(Q.cpu()),
           lambda: dsa.norm_rope(Q, out=(z(4, 8, 64), None)), lambda: dsa.norm_rope_bwd(Q, None, z(4, 7, 128), None)]
    kc, ic, table, lens = z(6, 16, 2, 128), z(6, 16, 64), i(4, 3), i(4)
    K, I, cu = z(4, 2, 128), z(4, 64), i(5)
    bad += [lambda: dsa.cache_append(K, K, I, kc, kc, ic, table, i(4), lens), lambda: dsa.cache_append(K, K, I, kc, kc, ic, table, cu, i(5)),
            lambda: dsa.cache_append(K, K, I, kc, kc[:5], ic, table, cu, lens), lambda: dsa.cache_append(K, K, I, kc, kc, ic[:, :8], table, cu, lens),
            lambda: dsa.cache_append(K, K[:3], I, kc, kc, ic, table, cu, lens), lambda: dsa.cache_append(K, K, I, kc[:, ::2], kc, ic, table, cu, lens),
            lambda: dsa.cache_append(K, K, I, kc, kc, ic, table[:, :2], cu, lens), lambda: dsa.cache_append(K, K, I, kc, kc, ic, table.long(), cu, lens)]
    q, w = z(4, 8, 64), z(4, 8)
    bad += [lambda: dsa.index_paged(q, ic, w[:3], table, lens, 48), lambda: dsa.index_paged(q[:3], ic, w, table, lens, 48),
            lambda: dsa.index_paged(q, ic, w, table, lens, 48, scores=z(3, 48, t=torch.float32)),
            lambda: dsa.index_paged(q, ic[..., :32], w, table, lens, 48)]
    idx = i(4, 16)
    bad += [lambda: dsa.sparse_attn_decode_paged(Q, kc, kc, idx[:3], table, lens), lambda: dsa.sparse_attn_decode_paged(Q[:3], kc, kc, idx, table, lens),
            lambda: dsa.sparse_attn_decode_paged(Q, kc, kc[..., :64], idx, table, lens),
            lambda: dsa.sparse_attn_decode_paged(Q, kc, kc, idx, table, lens, out=(z(4, 8, 64), None))]
    bad += [lambda: dsa.decode_paged(q, w, Q[:2], kc, kc, ic, table, lens, 48, 16),
            lambda: dsa.decode_paged(q, w, Q, kc, kc, ic, table, lens, 48, 16, out=(i(4, 32), z(4, 8, 128), None)),
            lambda: dsa.decode_step_paged(q, w, Q, K[:3], K, I, kc, kc, ic, table, lens, 48, 16)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(dsa.DSAError):  # a score row that max_seqlen_k does not fit in
        dsa.index_paged(q, ic, w, table, lens, 48, scores=z(4, 44, t=torch.float32))
    with pytest.raises(dsa.DSAError):
        dsa.decode_paged(q, w, Q, kc, kc, ic, table, lens, 48, 16, workspace=z(64, t=torch.uint8))


def test_binding_refuses_sizes_past_32_bits():
    """Sizes that the library takes in 32 bits are refused, not cut (tensors of no rows: no memory)."""
    z = lambda *s, t=BF16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    i = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    kc, ic, huge = z(6, 16, 2, 128), z(6, 16, 64), 2 ** 32 + 16
    bad = [lambda: dsa.sparse_attn_decode_paged(z(0, 8, 128), kc, kc, i(0, huge), i(0, 3), i(0)),
           lambda: dsa.sparse_attn_decode_paged(z(0, 8, 128), kc, kc, i(0, 16), i(0, huge), i(0)),
           lambda: dsa.index_paged(z(0, 8, 64), ic, z(0, 8), i(0, huge), i(0), 48),
           lambda: dsa.index_paged(z(0, 8, 64), ic, z(0, 8), i(0, 3), i(0), huge)]
    for call in bad:
        with pytest.raises(ValueError, match="32 bits"):
            call()
