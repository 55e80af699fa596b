"""The head norm and rotation and its gradients against plain 64-bit forms."""
import pytest
import torch

import lightning_indexer_b200 as dsa
import paged_testutil as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6


def randn(*shape, gen, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(torch.bfloat16)


def weight(d, gen):
    return (1 + 0.3 * torch.randn(d, generator=gen)).to(torch.bfloat16)


def dev(x):
    return None if x is None else x.cuda()


def check(got, want, tol, what):
    err = (ref.f64(got) - want).abs()
    assert bool((err <= tol).all()), f"{what}: off by {float((err - tol).max())} beyond its bound"


# T, Hq, Hk, d, rotary, interleaved: one row, one head, heads that do and do not fill a warp's
# rows, sizes past one group per warp
SHAPES = [(1, 1, 1, 128, 128, False), (1, 32, 4, 128, 128, False), (3, 5, 1, 64, 64, False), (17, 12, 3, 128, 64, True),
          (257, 7, 7, 32, 16, False), (66, 64, 1, 128, 64, True), (900, 32, 4, 128, 128, False), (4099, 20, 5, 64, 32, True),
          (130, 8, 2, 64, 0, False), (31, 3, 2, 32, 32, True)]


@pytest.mark.parametrize("T,Hq,Hk,d,rotary,inter", SHAPES)
@pytest.mark.parametrize("norm", [(True, True), (False, True), (False, False)])
def test_forward(T, Hq, Hk, d, rotary, inter, norm):
    g = torch.Generator().manual_seed(T * 7 + d)
    Q, K = randn(T, Hq, d, gen=g, scale=3.0), randn(T, Hk, d, gen=g, scale=0.05)
    gq, gk = (weight(d, g) if n else None for n in norm)
    freq = ref.frequencies(rotary) if rotary else None
    pos = torch.randint(0, 1_000_000, (T,), generator=g, dtype=torch.int32)
    Qo, Ko = dsa.norm_rope(Q.cuda(), K.cuda(), dev(gq), dev(gk), dev(freq), positions=pos.cuda(), interleaved=inter, eps=EPS)
    for got, x, w, what in ((Qo, Q, gq, "Q"), (Ko, K, gk, "K")):
        x, w = ref.f64(x), None if w is None else ref.f64(w)
        want = ref.norm_rope(x, w, EPS, pos, freq, inter)
        check(got, want, ref.norm_rope_tolerance(x, w, EPS, want), what)
    # without K
    alone, none = dsa.norm_rope(Q.cuda(), None, dev(gq), None, dev(freq), positions=pos.cuda(), interleaved=inter, eps=EPS)
    assert none is None and torch.equal(alone, Qo)


@pytest.mark.parametrize("given_lens", [False, True])
def test_packed_positions_and_rows_outside(given_lens):
    """Positions from the offsets; empty sequences; rows before the first and behind the last one."""
    g = torch.Generator().manual_seed(3)
    T, H, d = 50, 6, 64
    cu = torch.tensor([2, 2, 9, 10, 10, 43], dtype=torch.int32)
    lens = torch.tensor([0, 1000, 1, 5, 262144], dtype=torch.int32) if given_lens else None
    x = randn(T, H, d, gen=g)
    w, freq = weight(d, g), ref.frequencies(d)
    out = torch.full((T, H, d), 7.0, dtype=torch.bfloat16).cuda()
    dsa.norm_rope(x.cuda(), None, w.cuda(), None, freq.cuda(), cu_seqlens_q=cu.cuda(), seqlens_k=dev(lens), out=(out, None))
    pos = torch.zeros(T, dtype=torch.int64)
    for b in range(5):
        lo, hi = int(cu[b]), int(cu[b + 1])
        pos[lo:hi] = torch.arange(hi - lo) + (int(lens[b]) - (hi - lo) if given_lens else 0)
    want = ref.norm_rope(ref.f64(x), ref.f64(w), 1e-6, pos, freq, False)
    tol = ref.norm_rope_tolerance(ref.f64(x), ref.f64(w), 1e-6, want)
    check(out[2:43], want[2:43], tol[2:43], "rows of the sequences")
    assert bool((out[:2] == 7).all()) and bool((out[43:] == 7).all())
    # a row that belongs to no sequence takes no part in the weight's gradient either
    dy = randn(T, H, d, gen=g)
    cu_all = dict(cu_seqlens_q=cu.cuda(), seqlens_k=dev(lens))
    _, _, dg, _ = dsa.norm_rope_bwd(x.cuda(), None, dy.cuda(), None, w.cuda(), None, freq.cuda(), **cu_all)
    x2, dy2 = x.clone(), dy.clone()
    x2[:2], dy2[:2], x2[43:], dy2[43:] = 9.0, float("nan"), float("inf"), 5.0
    _, _, dg2, _ = dsa.norm_rope_bwd(x2.cuda(), None, dy2.cuda(), None, w.cuda(), None, freq.cuda(), **cu_all)
    assert torch.equal(dg, dg2)


def test_fused_projection_slices_and_in_place():
    g = torch.Generator().manual_seed(4)
    T, Hq, Hk, d = 37, 8, 2, 128
    x = randn(T, (Hq + 2 * Hk) * d, gen=g).cuda()
    before = x.clone()
    Q, K = x[:, :Hq * d].unflatten(1, (Hq, d)), x[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
    gq, gk, freq = weight(d, g).cuda(), weight(d, g).cuda(), ref.frequencies(d).cuda()
    Qo, Ko = dsa.norm_rope(Q, K, gq, gk, freq)
    assert torch.equal(x, before)
    Qd, Kd = dsa.norm_rope(Q.contiguous(), K.contiguous(), gq, gk, freq)
    assert torch.equal(Qo, Qd) and torch.equal(Ko, Kd)
    dsa.norm_rope(Q, K, gq, gk, freq, out=(Q, K))  # in the projection itself
    assert torch.equal(Q, Qd) and torch.equal(K, Kd)
    assert torch.equal(x[:, (Hq + Hk) * d:], before[:, (Hq + Hk) * d:])


def test_special_values():
    """A zero row stays zero; infinities and NaN stay in their own rows; negative positions turn back."""
    T, H, d = 9, 4, 64
    g = torch.Generator().manual_seed(5)
    x = randn(T, H, d, gen=g)
    x[0], x[1, 2, 5], x[2, 0, 0] = 0.0, float("nan"), float("inf")
    freq = ref.frequencies(d)
    pos = torch.tensor([5, 1, 2, -1, -70000, 0, 2 ** 31 - 1, 3, 4], dtype=torch.int32)
    y, _ = dsa.norm_rope(x.cuda(), None, torch.ones(d, dtype=torch.bfloat16).cuda(), None, freq.cuda(), positions=pos.cuda())
    y = y.cpu()
    assert bool((y[0] == 0).all()) and bool(y[1, 2].isnan().all()) and bool(y[2, 0].isnan().any())
    keep = torch.ones(T, H, dtype=torch.bool)
    keep[1, 2] = keep[2, 0] = False
    # position 2^31 - 1: its angle in turns, 3.4e8, is off by 3 * 2^-53 of itself, 1.2e-7 turns or 7e-7 rad
    want = ref.norm_rope(ref.f64(x), torch.ones(d).double(), 1e-6, pos, freq, False)
    tol = ref.norm_rope_tolerance(ref.f64(x), torch.ones(d).double(), 1e-6, want)
    tol[6] += 2e-6 * want[6].abs().amax()
    check(y[keep], want[keep], tol[keep], "rows without special values")


@pytest.mark.parametrize("T,Hq,Hk,d,rotary,inter", SHAPES)
@pytest.mark.parametrize("norm", [(True, True), (True, False), (False, True), (False, False)])
def test_backward(T, Hq, Hk, d, rotary, inter, norm):
    g = torch.Generator().manual_seed(T * 11 + d)
    Q, K = randn(T, Hq, d, gen=g, scale=2.0), randn(T, Hk, d, gen=g, scale=0.1)
    dQo, dKo = randn(T, Hq, d, gen=g, scale=0.2), randn(T, Hk, d, gen=g)
    gq, gk = (weight(d, g) if n else None for n in norm)
    freq = ref.frequencies(rotary) if rotary else None
    pos = torch.randint(0, 300_000, (T,), generator=g, dtype=torch.int32)
    args = (Q.cuda(), K.cuda(), dQo.cuda(), dKo.cuda(), dev(gq), dev(gk), dev(freq))
    dQ, dK, dgq, dgk = dsa.norm_rope_bwd(*args, positions=pos.cuda(), interleaved=inter, eps=EPS)
    for got, dw, x, dy, w, what in ((dQ, dgq, Q, dQo, gq, "Q"), (dK, dgk, K, dKo, gk, "K")):
        x, dy = ref.f64(x).requires_grad_(), ref.f64(dy)
        w = None if w is None else ref.f64(w).requires_grad_()
        ref.norm_rope(x, w, EPS, pos, freq, inter).backward(dy)
        dn = ref.rotate(dy, pos, freq, inter, -1.0)
        if w is None:
            assert dw is None
            check(got, x.grad, 2.0 ** -8 * x.grad.abs() + 3e-6 * dn.abs().amax(-1, keepdim=True), what)
            continue
        # fp32 before the rounding: dn * g is off by 3e-6 of the row's largest |dn g| (as forward); the
        # row's mean of dn g xh, a sum like the squares', by 3e-6 of that times mean |xh| <= 1; rstd and
        # xh by 1e-6: with M the largest |dn g| of the row, below rstd M (4e-6 + 5e-6 |xh|)
        xd = x.detach()
        rstd = torch.rsqrt(xd.pow(2).mean(-1, keepdim=True) + EPS)
        e, xh = (dn * w.detach()).abs().amax(-1, keepdim=True), (xd * rstd).abs()
        check(got, x.grad, 2.0 ** -8 * x.grad.abs() + rstd * e * (4e-6 + 5e-6 * xh), what)
        # the weight's gradient: terms off by 4e-6 of (|dn| row max) |xh|; summed in chains of at most
        # `iters` rows, then over row groups, 8 warps and blocks / 32 shares in 32 strands
        rows = T * x.shape[1]
        groups = (T * (Hq + Hk)) * d / 512 + 2
        chain = groups / (16 * 148) + 1 + 5 + 8 + (rows * d / 512 / 8 + 1) / 32 + 32
        bound = (dn.abs().amax(-1, keepdim=True) * xh).sum((0, 1)) * (4e-6 + chain * 2.0 ** -24)
        check(dw, w.grad, bound, what + " weight")
    again = dsa.norm_rope_bwd(*args, positions=pos.cuda(), interleaved=inter, eps=EPS)
    assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip((dQ, dK, dgq, dgk), again))


@pytest.mark.parametrize("inter", [False, True])
def test_backward_against_differences(inter):
    """The gradients along random directions against central differences of the 64-bit forward."""
    g = torch.Generator().manual_seed(6)
    T, H, d = 5, 3, 64
    x, dy, w = randn(T, H, d, gen=g), randn(T, H, d, gen=g), weight(d, g)
    freq, pos = ref.frequencies(32), torch.tensor([0, 1, 7, 4000, 250000], dtype=torch.int32)
    dx, _, dw, _ = dsa.norm_rope_bwd(x.cuda(), None, dy.cuda(), None, w.cuda(), None, freq.cuda(), positions=pos.cuda(), interleaved=inter)
    x, dy, w = ref.f64(x), ref.f64(dy), ref.f64(w)

    def loss(x, w):
        return (ref.norm_rope(x, w, 1e-6, pos, freq, inter) * dy).sum()

    h = 1e-5
    for _ in range(3):
        rx, rw = torch.randn(x.shape, generator=g).double(), torch.randn(d, generator=g).double()
        got = (ref.f64(dx) * rx).sum()
        want = (loss(x + h * rx, w) - loss(x - h * rx, w)) / (2 * h)
        # each element of dx is rounded by at most 2^-8 of itself; differences: h^2 and 64-bit noise / h
        assert abs(got - want) <= 2.0 ** -8 * (ref.f64(dx) * rx).abs().sum() * 1.01 + 1e-4
        got, want = (ref.f64(dw) * rw).sum(), (loss(x, w + h * rw) - loss(x, w - h * rw)) / (2 * h)
        assert abs(got - want) <= 1e-5 * (ref.f64(dw) * rw).abs().sum() + 1e-4


def test_backward_in_place_and_workspace():
    g = torch.Generator().manual_seed(8)
    T, Hq, Hk, d = 70, 4, 1, 128
    Q, K, dQo, dKo = (randn(T, h, d, gen=g).cuda() for h in (Hq, Hk, Hq, Hk))
    w, freq = weight(d, g).cuda(), ref.frequencies(d).cuda()
    a = dsa.norm_rope_bwd(Q, K, dQo, dKo, w, w, freq)
    ws = torch.full((dsa.norm_rope_bwd_workspace_bytes(T, Hq, Hk, d),), 255, dtype=torch.uint8, device="cuda")
    b = dsa.norm_rope_bwd(Q, K, dQo, dKo, w, w, freq, out=(dQo, dKo), workspace=ws)
    assert b[0] is dQo and all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(dsa.DSAError):
        dsa.norm_rope_bwd(Q, K, dQo, dKo, w, w, freq, workspace=ws[:-16])


def test_no_tokens():
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    Q, K = dsa.norm_rope(e, e, w, w)
    assert Q.shape == e.shape and K.shape == e.shape
    dQ, dK, dg, _ = dsa.norm_rope_bwd(e, e, e, e, w, None)
    assert dQ.shape == e.shape and bool((dg == 0).all())


def test_graph_and_streams():
    """A captured call replayed on new inputs, and calls on two streams at once."""
    g = torch.Generator().manual_seed(9)
    T, H, d = 300, 8, 128
    x, dy, w, freq = randn(T, H, d, gen=g).cuda(), randn(T, H, d, gen=g).cuda(), weight(d, g).cuda(), ref.frequencies(d).cuda()
    out = (torch.empty_like(x), None)
    dsa.norm_rope(x, None, w, None, freq, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.norm_rope(x, None, w, None, freq, out=out)
        grads = dsa.norm_rope_bwd(x, None, dy, None, w, None, freq)
    for seed in (1, 2):
        x.copy_(randn(T, H, d, gen=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], dsa.norm_rope(x, None, w, None, freq)[0])
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(grads, dsa.norm_rope_bwd(x, None, dy, None, w, None, freq)))
    want = dsa.norm_rope_bwd(x, None, dy, None, w, None, freq)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        with torch.cuda.stream(s):
            got.append([dsa.norm_rope_bwd(x, None, dy, None, w, None, freq) for _ in range(8)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for runs in got for r in runs for a, b in ((r[0], want[0]), (r[2], want[2])))


def test_dependent_calls_back_to_back():
    """A chain of calls, each on the last one's output, gives what it gives with the device waited for
    after every call."""
    g = torch.Generator().manual_seed(10)
    T, H, d = 2500, 8, 128
    x, w, f = randn(T, H, d, gen=g).cuda(), weight(d, g).cuda(), ref.frequencies(d).cuda()

    def chain(wait):
        y, z = x.clone(), torch.empty_like(x)
        for i in range(40):
            dsa.norm_rope(y, None, w, None, f, out=(z, None))
            if wait:
                torch.cuda.synchronize()
            y, _, dw, _ = dsa.norm_rope_bwd(z, None, y, None, w, None, f)
            if wait:
                torch.cuda.synchronize()
        return y, dw

    assert all(torch.equal(a, b) for a, b in zip(chain(False), chain(True)))
