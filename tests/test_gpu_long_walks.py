"""Sizes at which a block of the paged indexer goes round its ring of key stages several times, and a
warp of the norm-and-rotation backward walks several runs of rows."""
import pytest
import torch

import lightning_indexer_b200 as dsa
import paged_testutil as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
EPS = 1e-6


# The tiles of 128 positions are dealt to at most 148 blocks; a block has 6 key stages at d_I = 128, 12 at
# 64 and 16 at 32.  `times` makes that at least three rounds: 2921, 5839 and 7589 tiles, 19, 39 and 51 a block.
@pytest.mark.parametrize("H_I,d_I,times", [(64, 128, 1.0), (32, 128, 1.0), (16, 128, 1.0), (8, 64, 2.0), (4, 32, 2.6)])
@pytest.mark.parametrize("page", [16, 128, 1024])
def test_index_paged_rings(H_I, d_I, times, page):
    g = torch.Generator().manual_seed(H_I * 3 + page)
    lens = [int(n * times) for n in (150001, 7, 90000, 0, 100037, 33333)]
    B, N, pool = len(lens), max(lens), 4096 // page + 3  # pages are shared by all sequences
    # products of integers up to 8 and weights 1/2, 1/4, 1/8: every sum is exact in fp32
    q = torch.randint(-8, 9, (B, H_I, d_I), generator=g).to(BF16).cuda()
    cache = torch.randint(-8, 9, (pool, page, d_I), generator=g).to(BF16).cuda()
    w = (0.5 ** torch.randint(1, 4, (B, H_I), generator=g)).to(BF16).cuda()
    table = torch.randint(0, pool, (B, (N + page - 1) // page), generator=g, dtype=torch.int32)
    missing = torch.rand(table.shape, generator=g) < 0.02
    table[missing] = torch.where(torch.rand(int(missing.sum()), generator=g) < 0.5, -1, pool).to(torch.int32)
    table = table.cuda()
    scores = torch.full((B, (N + 3) // 4 * 4), 123.0, device="cuda")
    dsa.index_paged(q, cache, w, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), N, scores=scores)
    rows = torch.einsum("bhd,sd->bhs", q.double(), cache.flatten(0, 1).double()).clamp(min=0)
    rows = (w.double()[:, :, None] * rows).sum(1)  # [B, pool * page]
    for b, n in enumerate(lens):
        s = torch.arange(n, device="cuda")
        pages = table[b].long()[s // page]
        there = (pages >= 0) & (pages < pool)
        want = torch.where(there, rows[b][pages.clamp(0, pool - 1) * page + s % page], float("-inf"))
        assert torch.equal(scores[b, :n].double(), want), b
        assert bool((scores[b, n:] == 123.0).all())
    assert dsa.device_status() == (0, 0)


# T, Hq, Hk, d, rotary, interleaved, offsets: past 18944 groups of 512 / d rows a warp takes several runs;
# groups inside one token or over several, key tensors of one head (their runs are short), half rotated,
# a last run and a last group that are not full, tokens of no sequence at both ends
@pytest.mark.parametrize("T,Hq,Hk,d,rotary,inter,offsets", [
    (20011, 32, 4, 128, 128, False, [5, 7000, 7000, 20003]),
    (30011, 7, 1, 64, 64, False, [0, 11111, 30011]),
    (9001, 64, 1, 128, 64, True, [1, 9000]),
    (40009, 3, 5, 128, 128, True, [2, 40009]),
    (50021, 8, 2, 32, 16, False, [0, 50020]),
])
def test_backward_over_several_runs(T, Hq, Hk, d, rotary, inter, offsets):
    assert T * (Hq + Hk) * d / 512 > 18944
    g = torch.Generator(device="cuda").manual_seed(T)

    def rows(H, scale):
        return (torch.randn(T, H, d, generator=g, device="cuda") * scale).to(BF16)

    Q, K, dQo, dKo = rows(Hq, 2.0), rows(Hk, 0.1), rows(Hq, 0.2), rows(Hk, 1.0)
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(BF16) for _ in range(2))
    freq = ref.frequencies(rotary).cuda()
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    args = (Q, K, dQo, dKo, wq, wk, freq)
    got = dsa.norm_rope_bwd(*args, cu_seqlens_q=cu, interleaved=inter, eps=EPS)
    lo, hi = offsets[0], offsets[-1]
    pos = torch.cat([torch.arange(b - a, device="cuda") for a, b in zip(offsets, offsets[1:])])
    groups = T * (Hq + Hk) * d / 512
    for out, dw, x, dy, w in ((got[0], got[2], Q, dQo, wq), (got[1], got[3], K, dKo, wk)):
        assert bool((out[:lo] == 0).all()) and bool((out[hi:] == 0).all())
        x, dy, w = x[lo:hi].double().requires_grad_(), dy[lo:hi].double(), w.double().requires_grad_()
        ref.norm_rope(x, w, EPS, pos, freq, inter).backward(dy)
        # as for the short batches: fp32 before the one rounding, 3e-6 of the row's largest |dn g| for the
        # turned products, as much of the row's mean times |xh|, 1e-6 for rstd and xh
        with torch.no_grad():
            dn = ref.rotate(dy, pos, freq, inter, -1.0)
            rstd = torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
            e, xh = (dn * w).abs().amax(-1, keepdim=True), (x * rstd).abs()
            off = (out[lo:hi].double() - x.grad).abs() - 2.0 ** -8 * x.grad.abs() - rstd * e * (4e-6 + 5e-6 * xh)
            assert float(off.max()) <= 0.0
            # the weight's gradient: terms off by 4e-6 of |dn|'s row maximum times |xh|.  Sums: a warp takes its
            # share of the groups of 2368 warps, at most 1.4 of the mean by the costs it is dealt by, and a run
            # of 8 more; then 5 levels of lanes, 8 warps, 296 / 32 shares to a strand and 32 strands
            chain = 1.4 * groups / 2368 + 8 + 5 + 8 + 10 + 32
            bound = (dn.abs().amax(-1, keepdim=True) * xh).sum((0, 1)) * (4e-6 + chain * 2.0 ** -24)
            assert bool(((dw.double() - w.grad).abs() <= bound).all())
        del x, dy, dn, xh, off
    again = dsa.norm_rope_bwd(*args, cu_seqlens_q=cu, interleaved=inter, eps=EPS)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
