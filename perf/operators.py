"""The serving and training operators around sparse attention: what is measured of them.

Five kinds of call, each in a plain form (elementary torch operations) and as the library's call:
  norm_rope      RMS norm of every query and key head and the position rotation
  norm_rope_bwd  its gradients
  append         new keys, values and indexer keys into a paged cache, keys normed and rotated
  index          indexer scores of one query row per sequence over the paged indexer keys
  attend         attention of one query row per sequence over its selected positions in the paged cache
"""
import math

import torch

own = False

EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------------------- the cases
def listed():
    gqa = {"Hq": 32, "Hkv": 4, "d": 128}
    small = {"Hq": 8, "Hkv": 2, "d": 64}
    return [
        # one decode step of 16 sequences far into 256K contexts: Q and K sliced from the fused projection
        dict(name="rope_decode_16", op="norm_rope", T=16, rotary=128, interleaved=False, norm=True, fused=True, far=262144, **gqa),
        # the prompt of a 32K prefill, three packed sequences
        dict(name="rope_prefill_32k", op="norm_rope", T=32768, rotary=128, interleaved=False, norm=True, fused=True, far=0, **gqa),
        # the indexer's side of an odd prefill chunk: 64 query heads, one shared key, half the dims rotated, no norm
        dict(name="rope_indexer_chunk", op="norm_rope", T=8191, rotary=64, interleaved=True, norm=False, fused=False, far=0, Hq=64, Hkv=1, d=128),
        # a packed 64K training batch
        dict(name="rope_bwd_train_64k", op="norm_rope_bwd", T=65536, rotary=128, interleaved=False, norm=True, fused=False, far=0, **gqa),
        # the backward of a short batch of the small configuration
        dict(name="rope_bwd_small", op="norm_rope_bwd", T=1000, rotary=64, interleaved=False, norm=True, fused=True, far=0, **small),
        # one decode step: a new token for each of 16 sequences of up to 8K positions
        dict(name="append_decode_16", op="append", B=16, new=1, N=8192, page=64, d_I=128, rotary=128, norm=True, Hkv=4, d=128),
        # a prefill chunk of 8192 tokens for each of four sequences
        dict(name="append_prefill_32k", op="append", B=4, new=8192, N=12345, page=16, d_I=128, rotary=128, norm=True, Hkv=4, d=128),
        # the decode step at 256K context, 16 sequences
        dict(name="index_256k", op="index", B=16, N=262144, ragged=False, page=64, H_I=64, d_I=128),
        # a few short conversations, one of them empty
        dict(name="index_short", op="index", B=5, N=4001, ragged=True, page=16, H_I=32, d_I=128),
        # a full batch of unequal contexts
        dict(name="index_batch_64", op="index", B=64, N=16384, ragged=True, page=32, H_I=64, d_I=128),
        # attention of the decode step at 256K context, 2048 selected positions each
        dict(name="attend_256k", op="attend", B=16, N=262144, ragged=False, page=64, k=2048, **gqa),
        # one short sequence of the small configuration
        dict(name="attend_small", op="attend", B=1, N=1024, ragged=False, page=16, k=128, **small),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "index", "attend"])
    d = rng.choice([64, 128])
    Hq, Hkv = rng.choice([(32, 4), (20, 5), (8, 2), (40, 5), (8, 1)])
    rotary = rng.choice([d, d, d // 2, 16])
    norm = rng.random() < 0.7
    page = rng.choice([16, 32, 64, 128])
    if op in ("norm_rope", "norm_rope_bwd"):
        return dict(op=op, T=_log(rng, 1, 50000), rotary=rotary, interleaved=rng.random() < 0.5, norm=norm,
                    fused=rng.random() < 0.5, far=rng.choice([0, 0, 4096, 1000000]), Hq=Hq, Hkv=Hkv, d=d)
    if op == "append":
        B = _log(rng, 1, 64)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, 32768 // B)
        return dict(op=op, B=B, new=new, N=new + _log(rng, 1, 8192 // (1 + B // 8)), page=page, d_I=rng.choice([64, 128]),
                    rotary=min(rotary, 64), norm=norm, Hkv=Hkv, d=d)
    B = _log(rng, 1, 128)
    N = _log(rng, 1, min(262144, 2000000 // B))
    if op == "index":
        H_I, d_I = rng.choice([(64, 128), (64, 128), (32, 128), (16, 128), (8, 64), (4, 32)])
        return dict(op=op, B=B, N=N, ragged=rng.random() < 0.7, page=page, H_I=H_I, d_I=d_I)
    return dict(op=op, B=B, N=N, ragged=rng.random() < 0.7, page=page, k=16 * _log(rng, 1, 128), Hq=Hq, Hkv=Hkv, d=d)


# ------------------------------------------------------------------- lengths, by the case alone
def _kv_lens(case):
    """Cached positions of each sequence; where they are ragged, between N / 4 and N, and the second sequence is empty."""
    B, N = case["B"], case["N"]
    if not case.get("ragged", True):
        return [N] * B
    lens = [max(1, N - (b * 7919) % (3 * N // 4 + 1)) for b in range(B)]
    if B > 1 and case["op"] != "append":
        lens[1] = 0
    return [max(x, case.get("new", 0)) for x in lens]


def _packed(T):
    """Offsets of a packed batch of T rows: up to three sequences of unequal length."""
    a, b = T // 2, T // 2 + T // 3
    return sorted({0, a, b, T})


def work(case):
    op = case["op"]
    if op in ("norm_rope", "norm_rope_bwd"):
        n = case["T"] * (case["Hq"] + case["Hkv"]) * case["d"]
        passes, per = (2, 7) if op == "norm_rope" else (3, 15)
        return {"bytes": passes * n * 2 + 4 * case["T"], "flops": per * n}
    if op == "append":
        T = case["B"] * case["new"]
        n = T * (2 * case["Hkv"] * case["d"] + case["d_I"])
        return {"bytes": 2 * n * 2 + 4 * case["B"], "flops": 7 * T * (case["Hkv"] * case["d"] + case["d_I"])}
    lens = _kv_lens(case)
    if op == "index":
        total = sum(lens)
        return {"bytes": total * (case["d_I"] * 2 + 4) + case["B"] * case["H_I"] * (case["d_I"] + 1) * 2,
                "flops": total * case["H_I"] * (2 * case["d_I"] + 3)}
    sel = sum(min(case["k"], n) for n in lens)
    return {"bytes": sel * 2 * case["Hkv"] * case["d"] * 2 + case["B"] * (2 * case["Hq"] * case["d"] * 2 + 4 * case["Hq"] + 4 * case["k"]),
            "flops": sel * 4 * case["Hq"] * case["d"]}


# -------------------------------------------------------------------------------- inputs
def _inv_freq(rotary):
    i = torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda")
    return BASE ** (-i / rotary)


def _randn(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(scale)


def _weight(n, g):
    return (1 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16)


def _pages(case, lens, g):
    """A page table over a shuffled pool with a few pages that no sequence holds; unused entries are -1."""
    P, B = case["page"], case["B"]
    need = [(n + P - 1) // P for n in lens]
    width, total = max(max(need), 1), sum(need)
    pool = total + 3
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(need, device="cuda")
    first = torch.cumsum(n, 0) - n
    j = torch.arange(width, device="cuda")
    at = (first[:, None] + j[None, :]).clamp_(max=pool - 1)
    return torch.where(j[None, :] < n[:, None], perm[at], torch.full_like(perm[at], -1)), pool


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op in ("norm_rope", "norm_rope_bwd"):
        T, Hq, Hkv, d = case["T"], case["Hq"], case["Hkv"], case["d"]
        if case["fused"]:  # slices of one projection [T, (Hq + 2 Hkv) d]
            x = _randn((T, (Hq + 2 * Hkv) * d), g)
            s["Q"] = x[:, :Hq * d].unflatten(1, (Hq, d))
            s["K"] = x[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
        else:
            s["Q"], s["K"] = _randn((T, Hq, d), g), _randn((T, Hkv, d), g)
        s["gq"], s["gk"] = (_weight(d, g), _weight(d, g)) if case["norm"] else (None, None)
        s["inv_freq"] = _inv_freq(case["rotary"])
        s["positions"] = s["cu"] = None
        if case["far"]:
            s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        else:
            s["cu"] = torch.tensor(_packed(T), dtype=torch.int32, device="cuda")
        if op == "norm_rope_bwd":
            s["dQ"], s["dK"] = _randn((T, Hq, d), g, 0.1), _randn((T, Hkv, d), g, 0.1)
        return s
    lens = _kv_lens(case)
    s["table"], pool = _pages(case, lens, g)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["max"] = max(max(lens), 1)
    P = case["page"]
    if op == "append":
        T, Hkv, d, d_I = case["B"] * case["new"], case["Hkv"], case["d"], case["d_I"]
        s["K"], s["V"], s["k_idx"] = _randn((T, Hkv, d), g), _randn((T, Hkv, d), g), _randn((T, d_I), g)
        s["k_cache"], s["v_cache"] = _randn((pool, P, Hkv, d), g), _randn((pool, P, Hkv, d), g)
        s["k_idx_cache"] = _randn((pool, P, d_I), g)
        s["gk"], s["gi"] = (_weight(d, g), _weight(d_I, g)) if case["norm"] else (None, None)
        s["inv_freq"] = _inv_freq(case["rotary"])
        s["cu"] = torch.arange(0, T + 1, case["new"], dtype=torch.int32, device="cuda")
    elif op == "index":
        B, H_I, d_I = case["B"], case["H_I"], case["d_I"]
        s["q_idx"], s["k_idx_cache"] = _randn((B, H_I, d_I), g), _randn((pool, P, d_I), g)
        s["w"] = torch.softmax(torch.randn((B, H_I), generator=g, device="cuda"), 1).to(torch.bfloat16)
        s["scores"] = torch.full((B, (s["max"] + 3) // 4 * 4), float("-inf"), device="cuda")
    else:
        B, Hkv, d, k = case["B"], case["Hkv"], case["d"], case["k"]
        s["Q"] = _randn((B, case["Hq"], d), g)
        s["k_cache"], s["v_cache"] = _randn((pool, P, Hkv, d), g), _randn((pool, P, Hkv, d), g)
        # k of each sequence's positions, ascending, -1 in the unused slots
        r = torch.rand((B, s["max"]), generator=g, device="cuda")
        r.masked_fill_(torch.arange(s["max"], device="cuda")[None, :] >= s["lens"][:, None], 2.0)
        v, at = torch.topk(r, min(k, s["max"]), dim=1, largest=False)
        at = torch.where(v < 2.0, at, s["max"]).sort(1).values
        s["indices"] = torch.full((B, k), -1, dtype=torch.int32, device="cuda")
        s["indices"][:, :at.shape[1]] = torch.where(at < s["max"], at, -1).to(torch.int32)
    return s


# ---------------------------------------------------------------------------- plain forms
def _positions(s, T):
    if s["positions"] is not None:
        return s["positions"]
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    return t - s["cu"][torch.searchsorted(s["cu"], t, right=True) - 1]


def _cos_sin(pos, inv_freq):
    a = pos.to(torch.float64)[:, None] * inv_freq
    return a.cos().float()[:, None, :], a.sin().float()[:, None, :]


def _rotate(x, cos, sin, interleaved):
    r = 2 * cos.shape[-1]
    u, v = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    a, b = u * cos - v * sin, v * cos + u * sin
    y = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([y, x[..., r:]], -1)


def _normed(x, g):
    x = x.float()
    return x if g is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * g.float()


def _norm_bwd(x, g, dn):
    """dx and dg of the norm, from the gradient at its output."""
    if g is None:
        return dn.to(torch.bfloat16)
    x, g = x.float(), g.float()
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xhat = x * rstd
    dg = (dn * xhat).sum((0, 1), dtype=torch.float64).float()
    gd = dn * g
    return (rstd * (gd - xhat * (gd * xhat).mean(-1, keepdim=True))).to(torch.bfloat16), dg


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm_rope":
        cos, sin = _cos_sin(_positions(s, c["T"]), s["inv_freq"])
        return (_rotate(_normed(s["Q"], s["gq"]), cos, sin, c["interleaved"]).to(torch.bfloat16),
                _rotate(_normed(s["K"], s["gk"]), cos, sin, c["interleaved"]).to(torch.bfloat16))
    if op == "norm_rope_bwd":
        cos, sin = _cos_sin(_positions(s, c["T"]), s["inv_freq"])
        return (_norm_bwd(s["Q"], s["gq"], _rotate(s["dQ"].float(), cos, -sin, c["interleaved"])),
                _norm_bwd(s["K"], s["gk"], _rotate(s["dK"].float(), cos, -sin, c["interleaved"])))
    P = c["page"]
    if op == "append":
        t = torch.arange(c["B"] * c["new"], device="cuda")
        b = torch.searchsorted(s["cu"], t, right=True) - 1
        pos = s["lens"][b] - (s["cu"][b + 1] - t)  # the last new token sits at the last cached position
        slot = s["table"][b, pos // P].long() * P + pos % P
        cos, sin = _cos_sin(pos, s["inv_freq"])
        s["k_cache"].view(-1, c["Hkv"], c["d"])[slot] = _rotate(_normed(s["K"], s["gk"]), cos, sin, False).to(torch.bfloat16)
        s["v_cache"].view(-1, c["Hkv"], c["d"])[slot] = s["V"]
        s["k_idx_cache"].view(-1, c["d_I"])[slot] = _rotate(_normed(s["k_idx"][:, None], s["gi"]), cos, sin, False)[:, 0].to(torch.bfloat16)
        return s["k_cache"], s["v_cache"], s["k_idx_cache"]
    if op == "index":
        k = s["k_idx_cache"][s["table"].clamp(min=0)].flatten(1, 2)[:, :s["max"]].float()
        dots = torch.matmul(s["q_idx"].float(), k.transpose(1, 2)).clamp_(min=0)
        got = torch.matmul(s["w"].float()[:, None, :], dots)[:, 0]
        seen = torch.arange(s["max"], device="cuda")[None, :] < s["lens"][:, None]
        out = torch.full_like(s["scores"], float("-inf"))
        out[:, :s["max"]] = torch.where(seen, got, float("-inf"))
        return out
    at = s["indices"].clamp(min=0).long()
    slot = s["table"].gather(1, at // P).clamp(min=0).long() * P + at % P
    k = s["k_cache"].view(-1, c["Hkv"], c["d"])[slot].float().transpose(1, 2)  # [B, Hkv, k, d]
    v = s["v_cache"].view(-1, c["Hkv"], c["d"])[slot].float().transpose(1, 2)
    q = s["Q"].float().unflatten(1, (c["Hkv"], c["Hq"] // c["Hkv"]))
    x = torch.matmul(q, k.transpose(2, 3)) / math.sqrt(c["d"])
    x = torch.where((s["indices"] >= 0)[:, None, None, :], x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m > float("-inf"), m, 0.0)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return o.flatten(1, 2).to(torch.bfloat16), (m + torch.log(total)).flatten(1)


# --------------------------------------------------------------------- the library's calls
def _run_own(s):
    import lightning_indexer_b200 as dsa
    c = s["case"]
    op = c["op"]
    if op == "norm_rope":
        return dsa.norm_rope(s["Q"], s["K"], s["gq"], s["gk"], s["inv_freq"], positions=s["positions"], cu_seqlens_q=s["cu"],
                             interleaved=c["interleaved"], eps=EPS)
    if op == "norm_rope_bwd":
        dQ, dK, dgq, dgk = dsa.norm_rope_bwd(s["Q"], s["K"], s["dQ"], s["dK"], s["gq"], s["gk"], s["inv_freq"], positions=s["positions"],
                                             cu_seqlens_q=s["cu"], interleaved=c["interleaved"], eps=EPS)
        return ((dQ, dgq), (dK, dgk)) if c["norm"] else (dQ, dK)
    if op == "append":
        dsa.cache_append(s["K"], s["V"], s["k_idx"], s["k_cache"], s["v_cache"], s["k_idx_cache"], s["table"], s["cu"], s["lens"],
                         k_weight=s["gk"], k_idx_weight=s["gi"], inv_freq=s["inv_freq"], idx_inv_freq=s["inv_freq"], eps=EPS)
        return s["k_cache"], s["v_cache"], s["k_idx_cache"]
    if op == "index":
        return dsa.index_paged(s["q_idx"], s["k_idx_cache"], s["w"], s["table"], s["lens"], s["max"], scores=s["scores"])
    return dsa.sparse_attn_decode_paged(s["Q"], s["k_cache"], s["v_cache"], s["indices"], s["table"], s["lens"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------- the definitions in 64 bits, written apart
def _turned(x, pos, inv_freq, interleaved, sign=1.0):
    """x [T, H, d] in 64 bits with its first dims, taken as complex numbers, turned by sign * pos * inv_freq."""
    n = inv_freq.numel()
    a = sign * torch.outer(pos.double(), inv_freq)[:, None, :]
    z = torch.polar(torch.ones_like(a), a)
    y = x.clone()
    re = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    im = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    turned = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * z
    y[..., re], y[..., im] = turned.real, turned.imag
    return y


def _unit(x):
    return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm_rope", "norm_rope_bwd"):
        T = case["T"]
        pos = s["positions"]
        if pos is None:
            cu = _packed(T)
            pos = torch.cat([torch.arange(b - a, device="cuda") for a, b in zip(cu, cu[1:])])
        got = []
        for x, gw, name in ((s["Q"], s["gq"], "dQ"), (s["K"], s["gk"], "dK")):
            x = x.double()
            if op == "norm_rope":
                got.append(_turned(x if gw is None else _unit(x) * gw.double(), pos, s["inv_freq"], case["interleaved"]))
                continue
            dn = _turned(s[name].double(), pos, s["inv_freq"], case["interleaved"], -1.0)
            if gw is None:
                got.append(dn)
                continue
            # y = g x / r with r = sqrt(|x|^2 / d + eps):  dx = (g dn) / r - x ((g dn) . x) / (d r^3)
            r = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
            e = dn * gw.double()
            got.append((e / r - x * (e * x).sum(-1, keepdim=True) / (x.shape[-1] * r ** 3), (dn * x / r).flatten(0, 1).sum(0)))
        return tuple(got)
    lens, P = _kv_lens(case), case["page"]
    table = s["table"].tolist()
    if op == "append":
        new = case["new"]
        pos = torch.cat([torch.arange(n - new, n) for n in lens])
        slot = torch.cat([torch.tensor(table[b])[torch.arange(n - new, n) // P] * P + torch.arange(n - new, n) % P for b, n in enumerate(lens)]).cuda()
        pos = pos.cuda()
        out = []
        for x, cache, gw, turn in ((s["K"], s["k_cache"], s["gk"], True), (s["V"], s["v_cache"], None, False),
                                   (s["k_idx"][:, None], s["k_idx_cache"][:, :, None], s["gi"], True)):
            y = x.double()
            y = y if gw is None else _unit(y) * gw.double()
            y = _turned(y, pos, s["inv_freq"], False) if turn else y
            whole = cache.double()
            whole.flatten(0, 1).index_copy_(0, slot, y)
            out.append(whole)
        return out[0], out[1], out[2][:, :, 0]
    if op == "index":
        out = torch.full(s["scores"].shape, float("-inf"), dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            if n:
                k = s["k_idx_cache"][torch.tensor(table[b][:(n + P - 1) // P], device="cuda")].flatten(0, 1)[:n].double()
                out[b, :n] = (k @ s["q_idx"][b].double().T).relu() @ s["w"][b].double()
        return out
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    O = torch.zeros((case["B"], Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], Hq), float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        at = s["indices"][b][s["indices"][b] >= 0].long()
        if at.numel():
            rows = s["table"][b].long()[at // P], at % P
            k = s["k_cache"][rows].double().repeat_interleave(Hq // Hkv, 1)  # [n, Hq, d]
            v = s["v_cache"][rows].double().repeat_interleave(Hq // Hkv, 1)
            x = torch.einsum("hd,nhd->hn", s["Q"][b].double(), k) * d ** -0.5
            lse[b] = torch.logsumexp(x, 1)
            O[b] = torch.einsum("hn,nhd->hd", (x - lse[b][:, None]).exp(), v)
    return O, lse
