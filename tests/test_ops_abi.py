"""Argument checks of the operators around the losses: every refusal returns before
anything is enqueued, so no GPU is needed."""
import ctypes as C

import pytest

import catalogue_cross_entropy_amd as rece

P = C.c_void_p(1 << 20)   # never dereferenced
BIG = 1 << 40


def _embed_fwd(**kw):
    a = dict(n=100, C=50, d=64, dtype=1, table=P, ids=P, out=P)
    a.update(kw)
    return rece.lib().rece_embed_forward(None, a["n"], a["C"], a["d"], a["dtype"], 1.0, a["table"], a["ids"], a["out"])


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(C=0), 1), (dict(d=0), 1), (dict(d=12), 2), (dict(d=8200), 2), (dict(n=1 << 31), 2),
    (dict(C=1 << 31), 2), (dict(dtype=5), 2), (dict(table=None), 1), (dict(ids=None), 1), (dict(out=None), 1),
    (dict(table=C.c_void_p(24)), 1), (dict(ids=C.c_void_p(18)), 1), (dict(out=C.c_void_p(8)), 1),
])
def test_embed_forward_refuses(kw, status):
    assert _embed_fwd(**kw) == status
    assert rece.lib().rece_last_error().decode()


def test_embed_forward_of_no_rows_is_nothing():
    assert _embed_fwd(n=0, table=None, ids=None, out=None) == 0


def _embed_bwd(**kw):
    a = dict(n=100, C=50, d=64, dtype=1, flags=0, ids=P, dout=P, ws=P, wsb=BIG, dtable=P)
    a.update(kw)
    return rece.lib().rece_embed_backward(None, a["n"], a["C"], a["d"], a["dtype"], 1.0, a["flags"], a["ids"], a["dout"],
                                          a["ws"], a["wsb"], a["dtable"])


@pytest.mark.parametrize("kw,status", [
    (dict(flags=1), 1), (dict(flags=8 | 16), 2), (dict(dtable=None), 1), (dict(ids=None), 1), (dict(dout=None), 1),
    (dict(ws=None), 1), (dict(wsb=16), 3), (dict(d=4), 2), (dict(dtype=2), 2), (dict(dtable=C.c_void_p(40)), 1),
    (dict(ws=C.c_void_p(40)), 1),
])
def test_embed_backward_refuses(kw, status):
    assert _embed_bwd(**kw) == status


def _lp_bytes(flags=0, **kw):
    a = dict(s=100, C=50, d=64, dtype=1)
    a.update(kw)
    n = C.c_size_t()
    return rece.lib().rece_logprob_workspace_bytes(a["s"], a["C"], a["d"], a["dtype"], flags, C.byref(n)), n.value


def _lp_fwd(**kw):
    a = dict(s=100, C=50, d=64, dtype=1, T=1.0, flags=0, X=P, Y=P, ids=P, ws=P, wsb=BIG, logp=P, ent=None)
    a.update(kw)
    return rece.lib().rece_logprob_forward(None, a["s"], a["C"], a["d"], a["dtype"], a["T"], a["flags"], a["X"], a["Y"],
                                           a["ids"], a["ws"], a["wsb"], a["logp"], a["ent"])


def _lp_bwd(**kw):
    a = dict(flags=0, dlogp=P, dent=None, dX=P, dY=P, T=1.0, wsb=BIG)
    a.update(kw)
    return rece.lib().rece_logprob_backward(None, 100, 50, 64, 1, a["T"], a["flags"], P, P, P, P, a["wsb"], a["dlogp"],
                                            a["dent"], a["dX"], a["dY"])


@pytest.mark.parametrize("kw,status", [
    (dict(s=0), 1), (dict(C=0), 1), (dict(d=48), 2), (dict(dtype=3), 2), (dict(s=1 << 31), 2), (dict(T=0.0), 1),
    (dict(T=-1.0), 1), (dict(T=float("nan")), 1), (dict(T=float("inf")), 1), (dict(flags=1), 1), (dict(flags=16), 1),
    (dict(X=None), 1), (dict(Y=None), 1), (dict(ids=None), 1), (dict(ws=None), 1), (dict(wsb=100), 3),
    (dict(logp=None), 1), (dict(ent=P), 1), (dict(flags=64), 1), (dict(X=C.c_void_p(8)), 1), (dict(ws=C.c_void_p(8)), 1),
])
def test_logprob_forward_refuses(kw, status):
    assert _lp_fwd(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(flags=32), 1), (dict(dlogp=None), 1), (dict(dX=None), 1), (dict(dY=None), 1), (dict(dent=P), 1),
    (dict(dX=C.c_void_p(4)), 1), (dict(wsb=100), 3), (dict(T=0.0), 1),
])
def test_logprob_backward_refuses(kw, status):
    assert _lp_bwd(**kw) == status


def test_logprob_workspace_holds_no_logits():
    """Far below s x C at every size, smaller without a backward call, and the same for equal arguments."""
    for s, c, d in ((1, 1, 32), (5, 1_000_000, 64), (51200, 30000, 64), (4099, 50021, 256), (2047, 200_000, 128)):
        for dtype in (0, 1):
            st, full = _lp_bytes(s=s, C=c, d=d, dtype=dtype)
            st2, fwd = _lp_bytes(flags=32, s=s, C=c, d=d, dtype=dtype)
            assert st == st2 == 0 and 0 < fwd <= full
            es = 4 if dtype == 0 else 2
            # packed rows and per-row scalars, and the parts of split sweeps (at most 256 MB each way,
            # or one part)
            rows = (s + 256) * (d * es + 64)
            assert full <= 2 * rows + max(256 << 20, 4 * d * max(s + 256, c)) + (12 << 20) + 4096 * 12 * 256


def _policy(n=100, n_seq=5, dtype=0, reduction=0, token=0, low=0.2, high=0.2, kl=0.0, ent=0.0):
    return rece.PolicyConfig(n, n_seq, dtype, reduction, token, low, high, kl, ent)


def _pol(cfg, **kw):
    a = dict(logp=P, old=P, ref=None, ent=None, adv=P, offs=P, mask=None, dloss=None, ws=P, wsb=BIG, loss=P, stats=P, dlogp=P,
             dent=None)
    a.update(kw)
    return rece.lib().rece_policy_loss(C.byref(cfg) if cfg else None, None, a["logp"], a["old"], a["ref"], a["ent"], a["adv"],
                                       a["offs"], a["mask"], a["dloss"], a["ws"], a["wsb"], a["loss"], a["stats"], a["dlogp"],
                                       a["dent"])


@pytest.mark.parametrize("cfg,status", [
    (dict(n=-1), 1), (dict(n_seq=0), 1), (dict(n=1 << 31), 2), (dict(dtype=2), 2), (dict(reduction=2), 1), (dict(token=2), 1),
    (dict(low=-0.1), 1), (dict(low=1.1), 1), (dict(high=-0.1), 1), (dict(high=float("inf")), 1), (dict(low=float("nan")), 1),
    (dict(kl=float("nan")), 1), (dict(ent=float("inf")), 1),
])
def test_policy_config_refused(cfg, status):
    n = C.c_size_t()
    c = _policy(**cfg)
    assert rece.lib().rece_policy_workspace_bytes(C.byref(c), C.byref(n)) == status
    assert _pol(c) == status


@pytest.mark.parametrize("cfg,kw,status", [
    (None, {}, 1), ({}, dict(logp=None), 1), ({}, dict(old=None), 1), ({}, dict(adv=None), 1), ({}, dict(offs=None), 1),
    ({}, dict(ws=None), 1), ({}, dict(loss=None), 1), ({}, dict(stats=None), 1), (dict(kl=0.1), {}, 1),
    (dict(ent=0.1), {}, 1), ({}, dict(dent=P), 1), (dict(n=1 << 20), dict(wsb=64), 3), ({}, dict(logp=C.c_void_p(2)), 1),
    ({}, dict(offs=C.c_void_p(2)), 1), (dict(dtype=1), dict(logp=C.c_void_p(3)), 1), ({}, dict(ws=C.c_void_p(8)), 1),
])
def test_policy_call_refused(cfg, kw, status):
    assert _pol(None if cfg is None else _policy(**cfg), **kw) == status


def _pref_cfg(n=100, n_seq=10, G=5, dtype=0, kind=0, average=0, beta=0.1, margin=0.0, smoothing=0.0):
    return rece.PreferenceConfig(n, n_seq, G, dtype, kind, average, beta, margin, smoothing)


def _pref(cfg, **kw):
    a = dict(logp=P, ref=None, offs=P, goffs=P, mask=None, dloss=None, ws=P, wsb=BIG, loss=P, pg=P, rewards=P, dlogp=P)
    a.update(kw)
    return rece.lib().rece_preference_loss(C.byref(cfg) if cfg else None, None, a["logp"], a["ref"], a["offs"], a["goffs"],
                                           a["mask"], a["dloss"], a["ws"], a["wsb"], a["loss"], a["pg"], a["rewards"],
                                           a["dlogp"])


@pytest.mark.parametrize("cfg,status", [
    (dict(n=-1), 1), (dict(n_seq=0), 1), (dict(G=0), 1), (dict(n=1 << 31), 2), (dict(dtype=2), 2), (dict(kind=4), 1),
    (dict(kind=-1), 1), (dict(average=2), 1), (dict(beta=0.0), 1), (dict(beta=float("nan")), 1), (dict(margin=float("inf")), 1),
    (dict(smoothing=1.0), 1), (dict(smoothing=-0.1), 1), (dict(kind=3, smoothing=0.1), 1),
])
def test_preference_config_refused(cfg, status):
    n = C.c_size_t()
    c = _pref_cfg(**cfg)
    assert rece.lib().rece_preference_workspace_bytes(C.byref(c), C.byref(n)) == status
    assert _pref(c) == status


@pytest.mark.parametrize("cfg,kw,status", [
    (None, {}, 1), ({}, dict(logp=None), 1), ({}, dict(offs=None), 1), ({}, dict(goffs=None), 1), ({}, dict(ws=None), 1),
    ({}, dict(loss=None), 1), ({}, dict(pg=None), 1), ({}, dict(rewards=None), 1), ({}, dict(wsb=4), 3),
    ({}, dict(ref=C.c_void_p(6)), 1), ({}, dict(goffs=C.c_void_p(6)), 1),
])
def test_preference_call_refused(cfg, kw, status):
    assert _pref(None if cfg is None else _pref_cfg(**cfg), **kw) == status


def test_python_options_refused():
    with pytest.raises(ValueError):
        rece.LogProb(10, 20, 64, temperature=0.0)
    with pytest.raises(ValueError):
        rece.LogProb(10, 20, 64, dtype="f16")
    with pytest.raises(ValueError):
        rece.PolicyLoss(10, 2, reduction="batch")
    with pytest.raises(ValueError):
        rece.PreferenceLoss(10, 2, 1, kind="other")
    with pytest.raises(rece.ReceError):
        rece.ItemEmbedding(10, 20, 12)
    with pytest.raises(rece.ReceError):
        rece.LogProb(10, 20, 80)


def test_python_tensors_refused():
    """Shapes, types, devices and missing companions are refused before the library is called."""
    import torch
    cpu = torch.zeros(10, 64, dtype=torch.bfloat16)
    ids = torch.zeros(10, dtype=torch.int32)
    with pytest.raises(ValueError):
        rece.ItemEmbedding(10, 10, 64).forward(cpu, ids)
    with pytest.raises(ValueError):
        rece.LogProb(10, 10, 64).forward(cpu, cpu, ids)
    with pytest.raises(ValueError):
        rece.PreferenceLoss(10, 2, 1).forward(ids.float(), None, ids, ids)
    with pytest.raises(ValueError):
        rece.PolicyLoss(10, 2).forward(ids.float(), ids.float(), ids.float(), ids)
