"""New outputs of the head norm and rotation and of its gradients hold zeros in the rows of tokens
that belong to no sequence; given ones keep what they held there."""
import pytest
import torch

import lightning_indexer_b200 as dsa
import paged_testutil as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def poison(*shapes):
    """Leaves NaN in the memory that the next tensors of these shapes are made of."""
    held = [torch.full(s, float("nan"), dtype=BF16, device="cuda") for s in shapes for _ in range(4)]
    torch.cuda.synchronize()
    del held


# T, Hq, Hk, d, rotary, interleaved, weights, offsets: rows that share their token or do not, with every
# dim rotated or half of them, no sequence at all, rows before the first one only, and sizes at which a
# warp of the backward walks several runs
CASES = [
    (50, 32, 4, 128, 128, False, True, [2, 2, 9, 10, 10, 43]),
    (50, 5, 1, 64, 64, False, True, [0, 20, 31]),
    (333, 7, 3, 32, 16, True, True, [100, 333]),
    (61, 8, 2, 64, 0, False, False, [7, 7]),
    (130, 64, 1, 128, 64, True, False, [0, 129]),
    (20011, 32, 4, 128, 128, False, True, [3, 9000, 9000, 15002]),
    (30011, 7, 1, 64, 32, False, True, [1000, 2000, 30010]),
]


@pytest.mark.parametrize("T,Hq,Hk,d,rotary,inter,norm,offsets", CASES)
def test_rows_outside_the_sequences(T, Hq, Hk, d, rotary, inter, norm, offsets):
    g = torch.Generator().manual_seed(T + d)

    def rows(H):
        return torch.randn(T, H, d, generator=g).to(BF16).cuda()

    Q, K, dQo, dKo = rows(Hq), rows(Hk), rows(Hq), rows(Hk)
    w = torch.linspace(0.5, 1.5, d).to(BF16).cuda() if norm else None
    freq = ref.frequencies(rotary).cuda() if rotary else None
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    lo, hi = offsets[0], offsets[-1]

    def calls(q_out, k_out):
        out = None if q_out is None else (q_out, k_out)
        return (lambda: dsa.norm_rope(Q, K, w, w, freq, cu_seqlens_q=cu, interleaved=inter, out=out),
                lambda: dsa.norm_rope_bwd(Q, K, dQo, dKo, w, w, freq, cu_seqlens_q=cu, interleaved=inter, out=out))

    for i in range(2):
        given = torch.full_like(Q, 7.0), torch.full_like(K, 7.0)
        kept = calls(*given)[i]()
        poison(Q.shape, K.shape)
        fresh = calls(None, None)[i]()
        for new, old in zip(fresh[:2], kept[:2]):
            assert bool((new[:lo] == 0).all()) and bool((new[hi:] == 0).all())
            assert bool((old[:lo] == 7).all()) and bool((old[hi:] == 7).all())
            assert torch.equal(new[lo:hi], old[lo:hi])
        for a, b in zip(fresh[2:], kept[2:]):  # the weights' gradients
            assert (a is None and b is None) or torch.equal(a, b)
    # without K, captured, and replayed over memory that holds NaN
    dsa.norm_rope(Q, None, w, None, freq, cu_seqlens_q=cu, interleaved=inter)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = dsa.norm_rope(Q, None, w, None, freq, cu_seqlens_q=cu, interleaved=inter)
        dx = dsa.norm_rope_bwd(Q, None, dQo, None, w, None, freq, cu_seqlens_q=cu, interleaved=inter)[0]
    y.fill_(float("nan"))
    dx.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for x in (y, dx):
        assert bool((x[:lo] == 0).all()) and bool((x[hi:] == 0).all()) and not bool(x.isnan().any())


def test_no_key_heads():
    """K of no heads: its outputs are empty and its weight's gradient, a sum over no rows, is zero."""
    Q = torch.ones(5, 4, 64, dtype=BF16, device="cuda")
    K, w = Q[:, :0], torch.ones(64, dtype=BF16, device="cuda")
    held = [torch.full((64,), float("nan"), device="cuda") for _ in range(200)]
    torch.cuda.synchronize()
    del held
    dQ, dK, dgq, dgk = dsa.norm_rope_bwd(Q, K, Q, K, w, w)
    want = dsa.norm_rope_bwd(Q, None, Q, None, w, None)
    assert dK.shape == K.shape and torch.equal(dQ, want[0]) and torch.equal(dgq, want[2])
    assert bool((dgk == 0).all())
