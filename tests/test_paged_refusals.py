"""What the head norm and rotation and the paged-cache calls refuse, on the CPU: the C ABI with
pointers that are never dereferenced, and the binding's checks of sizes."""
import pytest
import torch

import lightning_indexer_b200 as dsa
from lightning_indexer_b200 import _lib

FAKE = 1 << 20
MIS = FAKE + 2
BAD_ARG, UNSUPPORTED, WORKSPACE = -1, -2, -3


def refused(name, base, order, cases):
    """Each case changes some of the base arguments and names the status it must return."""
    fn = getattr(_lib.load(), name)
    for change, status in cases:
        args = {**base, **change}
        assert fn(*[args[n] for n in order], None) == status, (name, change)


ROPE = dict(Q=FAKE, qs=4096, K=FAKE, ks=512, gq=FAKE, gk=FAKE, eps=1e-6, freq=FAKE, rotary=128, inter=0, pos=None, cu=FAKE, lens=None,
            batch=2, T=8, Hq=32, Hk=4, d=128, Qo=FAKE, qos=4096, Ko=FAKE, kos=512)
ROPE_CASES = [
    (dict(Q=None), BAD_ARG), (dict(Q=MIS), BAD_ARG), (dict(K=MIS), BAD_ARG), (dict(gq=MIS), BAD_ARG), (dict(T=-1), BAD_ARG),
    (dict(K=None), BAD_ARG), (dict(Hk=0), BAD_ARG), (dict(Hq=0), BAD_ARG), (dict(qs=4095), BAD_ARG), (dict(qs=4100), BAD_ARG),
    (dict(ks=504), BAD_ARG), (dict(eps=-1.0), BAD_ARG), (dict(eps=float("nan")), BAD_ARG), (dict(rotary=0), BAD_ARG),
    (dict(freq=None), BAD_ARG), (dict(rotary=144), BAD_ARG), (dict(rotary=-16), BAD_ARG), (dict(cu=None), BAD_ARG), (dict(batch=0), BAD_ARG),
    (dict(cu=None, batch=1, lens=FAKE), BAD_ARG), (dict(rotary=24), UNSUPPORTED), (dict(d=96, rotary=96), UNSUPPORTED),
    (dict(T=1 << 27), UNSUPPORTED), (dict(qs=1 << 31), BAD_ARG), (dict(T=0), 0)]


def test_norm_rope_refusals():
    order = list(ROPE)
    refused("dsa_norm_rope", ROPE, order, ROPE_CASES + [(dict(Qo=None), BAD_ARG), (dict(Ko=MIS), BAD_ARG), (dict(qos=8), BAD_ARG)])


def test_norm_rope_bwd_refusals():
    lib = _lib.load()
    need = lib.dsa_norm_rope_bwd_workspace_size(8, 32, 4, 128)
    assert need > 0
    for bad in ((-1, 32, 4, 128), (8, 0, 4, 128), (8, 32, -1, 128), (8, 32, 4, 96)):
        assert lib.dsa_norm_rope_bwd_workspace_size(*bad) == 0
    base = dict(ROPE, dQo=FAKE, dqos=4096, dKo=FAKE, dkos=512, dQ=FAKE, dqs=4096, dK=FAKE, dks=512, dgq=FAKE, dgk=FAKE, ws=FAKE, nws=need)
    order = ["Q", "qs", "K", "ks", "dQo", "dqos", "dKo", "dkos", "gq", "gk", "eps", "freq", "rotary", "inter", "pos", "cu", "lens", "batch",
             "T", "Hq", "Hk", "d", "dQ", "dqs", "dK", "dks", "dgq", "dgk", "ws", "nws"]
    cases = [c for c in ROPE_CASES if c[1] != 0] + [
        (dict(dQo=None), BAD_ARG), (dict(dK=MIS), BAD_ARG), (dict(dqs=8), BAD_ARG), (dict(dgq=None), BAD_ARG), (dict(dgk=None), BAD_ARG),
        (dict(ws=None), WORKSPACE), (dict(ws=MIS), WORKSPACE), (dict(nws=need - 4), WORKSPACE)]
    refused("dsa_norm_rope_bwd", base, order, cases)


def test_norm_rope_bwd_workspace_follows_from_the_sizes():
    """A share of d sums for each block, at most 296 blocks, whatever device is current (or none)."""
    size = _lib.load().dsa_norm_rope_bwd_workspace_size
    for T, Hq, Hk, d in ((65536, 32, 4, 128), (1 << 20, 64, 1, 64), (40000, 32, 0, 128)):
        assert size(T, Hq, Hk, d) == 296 * d * 4
    assert 0 < size(1, 1, 0, 32) <= size(1000, 8, 2, 64) <= 296 * 64 * 4


@pytest.mark.parametrize("name", ["dsa_norm_rope_zeroed", "dsa_norm_rope_bwd_zeroed"])
def test_zeroed_forms_refuse_the_same(name, monkeypatch):
    lib, plain = _lib.load(), name.removesuffix("_zeroed")
    monkeypatch.setattr(lib, plain, getattr(lib, name))
    test_norm_rope_refusals() if plain == "dsa_norm_rope" else test_norm_rope_bwd_refusals()


POOL = dict(table=FAKE, width=8, lens=FAKE, batch=2, pages=16, page=16)
POOL_CASES = [(dict(table=None), BAD_ARG), (dict(lens=None), BAD_ARG), (dict(width=0), BAD_ARG), (dict(batch=0), BAD_ARG),
              (dict(pages=0), BAD_ARG), (dict(page=0), BAD_ARG), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
              (dict(page=2048), UNSUPPORTED), (dict(pages=1 << 27), UNSUPPORTED)]
BIG = 1 << 30  # page strides large enough for every page size of the cases


def test_cache_append_refusals():
    base = dict(K=FAKE, ks=512, V=FAKE, vs=512, I=FAKE, is_=128, gk=None, gi=None, eps=1e-6, freq=FAKE, rotary=128, inter=0, ifreq=FAKE,
                irotary=64, iinter=0, pos=None, cu=FAKE, T=8, Hkv=4, d=128, d_I=128, kc=FAKE, kcs=BIG, vc=FAKE, vcs=BIG, ic=FAKE, ics=BIG, **POOL)
    cases = POOL_CASES + [
        (dict(K=None), BAD_ARG), (dict(V=MIS), BAD_ARG), (dict(cu=None), BAD_ARG), (dict(T=-1), BAD_ARG), (dict(I=None), BAD_ARG),
        (dict(d_I=0), BAD_ARG), (dict(ic=None), BAD_ARG), (dict(kcs=16 * 512 - 8), BAD_ARG), (dict(vcs=16 * 512 + 4), BAD_ARG),
        (dict(ics=16 * 128 - 8), BAD_ARG), (dict(ks=504), BAD_ARG), (dict(is_=120), BAD_ARG), (dict(gk=MIS), BAD_ARG), (dict(irotary=0), BAD_ARG),
        (dict(irotary=144), BAD_ARG), (dict(eps=-0.5), BAD_ARG), (dict(irotary=24), UNSUPPORTED), (dict(d=80, rotary=80), UNSUPPORTED),
        (dict(d_I=48, irotary=48), UNSUPPORTED), (dict(T=0), 0),
        (dict(T=0, I=None, d_I=0, ic=None, ics=0, ifreq=None, irotary=0), 0)]
    refused("dsa_cache_append", base, list(base), cases)


def test_index_paged_refusals():
    base = dict(q=FAKE, ic=FAKE, ics=BIG, w=FAKE, table=FAKE, width=8, lens=FAKE, batch=2, pages=16, page=16, maxk=128, H_I=64, d_I=128,
                scores=FAKE, ld=128)
    cases = POOL_CASES + [(dict(q=None), BAD_ARG), (dict(w=MIS), BAD_ARG), (dict(ic=None), BAD_ARG), (dict(ics=16 * 128 - 8), BAD_ARG),
                          (dict(maxk=-1), BAD_ARG), (dict(scores=None), BAD_ARG), (dict(scores=MIS), BAD_ARG), (dict(ld=124), BAD_ARG),
                          (dict(ld=130), BAD_ARG), (dict(maxk=0x7FFFFFFF, ld=1 << 31), UNSUPPORTED), (dict(H_I=48), UNSUPPORTED), (dict(d_I=64), UNSUPPORTED)]
    refused("dsa_index_paged", base, list(base), cases)


def test_sparse_attn_decode_paged_refusals():
    base = dict(Q=FAKE, kc=FAKE, kcs=BIG, vc=FAKE, vcs=BIG, idx=FAKE, table=FAKE, width=8, lens=FAKE, batch=2, pages=16, page=16, Hq=32, Hkv=4,
                d=128, k=64, scale=0.1, O=FAKE, lse=None)
    cases = POOL_CASES + [(dict(Q=MIS), BAD_ARG), (dict(kc=None), BAD_ARG), (dict(vcs=16 * 512 - 8), BAD_ARG), (dict(idx=None), BAD_ARG),
                          (dict(O=None), BAD_ARG), (dict(k=0), BAD_ARG), (dict(scale=0.0), BAD_ARG), (dict(scale=float("nan")), BAD_ARG),
                          (dict(k=40), UNSUPPORTED), (dict(k=4112), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(Hq=12), UNSUPPORTED),
                          (dict(Hq=30), UNSUPPORTED)]
    refused("dsa_sparse_attn_decode_paged", base, list(base), cases)


def test_paged_pipeline_refusals():
    lib = _lib.load()
    need = lib.dsa_decode_paged_workspace_size(2, 128)
    assert need >= 2 * 128 * 4 and lib.dsa_decode_paged_workspace_size(0, 128) == 0 and lib.dsa_decode_paged_workspace_size(2, -1) == 0
    base = dict(qi=FAKE, w=FAKE, Q=FAKE, kc=FAKE, kcs=BIG, vc=FAKE, vcs=BIG, ic=FAKE, ics=BIG, table=FAKE, width=8, lens=FAKE, batch=2, pages=16,
                page=16, maxk=128, Hq=32, Hkv=4, d=128, H_I=64, d_I=128, k=64, scale=0.1, idx=FAKE, O=FAKE, lse=None, ws=FAKE, nws=need)
    pool = [c for c in POOL_CASES if c[1] != WORKSPACE]
    cases = pool + [(dict(qi=None), BAD_ARG), (dict(Q=MIS), BAD_ARG), (dict(idx=None), BAD_ARG), (dict(k=40), UNSUPPORTED),
                    (dict(H_I=48), UNSUPPORTED), (dict(maxk=1 << 30), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws=MIS), WORKSPACE),
                    (dict(nws=need - 1), WORKSPACE)]
    refused("dsa_decode_paged", base, list(base), cases)
    step_need = lib.dsa_decode_step_paged_workspace_size(2, 128, 32, 128, 64, 128)
    assert step_need >= need + 2 * (32 + 64) * 128 * 2
    step = dict(qi=FAKE, qis=8192, w=FAKE, Q=FAKE, qs=4096, K=FAKE, ks=512, V=FAKE, vs=512, I=FAKE, is_=128, gq=None, gk=None, gqi=None, gki=None,
                eps=1e-6, freq=FAKE, rotary=128, inter=0, ifreq=FAKE, irotary=64, iinter=0, pos=None)
    step.update({n: v for n, v in base.items() if n not in step})
    step["nws"] = step_need
    cases = pool + [(dict(I=None), BAD_ARG), (dict(qs=4088), BAD_ARG), (dict(qis=8190), BAD_ARG), (dict(gqi=MIS), BAD_ARG), (dict(k=40), UNSUPPORTED),
                    (dict(rotary=24), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(nws=step_need - 1), WORKSPACE)]
    refused("dsa_decode_step_paged", step, list(step), cases)


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.norm_rope(x)
    with pytest.raises(ValueError, match="bfloat16"):
        dsa.norm_rope(x.float())
    with pytest.raises(ValueError, match="CUDA"):
        dsa.norm_rope_bwd(x, None, x, None)
    cache = torch.zeros((3, 16, 4, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.cache_append(x, x, None, cache, cache, None, table, torch.zeros(3, dtype=torch.int32), lens)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.sparse_attn_decode_paged(x, cache, cache, torch.zeros((2, 16), dtype=torch.int32), table, lens)
    with pytest.raises(ValueError, match="CUDA"):
        dsa.index_paged(x, cache[:, :, 0], torch.zeros((2, 4), dtype=torch.bfloat16), table, lens, 16)


def test_missing_native_binding_fails_loudly(monkeypatch):
    import sys
    monkeypatch.setattr(dsa, "_native_module", None)
    monkeypatch.delattr(dsa, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, "lightning_indexer_b200._binding", None)
    with pytest.raises(ImportError):
        dsa.norm_rope(torch.zeros((1, 1, 32), dtype=torch.bfloat16))
