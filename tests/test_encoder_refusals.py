"""Argument checks of the sequence encoder's operators: every refusal returns before anything is enqueued, so no GPU is
needed.  And the bounds of log_buckets."""
import ctypes as C
import math

import pytest
import torch

import catalogue_cross_entropy_amd as rece

P = C.c_void_p(1 << 20)   # never dereferenced
BIG = 1 << 40


def config(**kw):
    a = dict(n=100, n_seq=3, q_stride=128, k_stride=64, v_stride=64, heads=4, kv_heads=2, d=32, dtype=1, scale=0.2, bounds=())
    a.update(kw)
    b = a.pop("bounds")
    count = a.pop("n_bounds", len(b))
    return rece.AttentionConfig(*(a[k] for k in ("n", "n_seq", "q_stride", "k_stride", "v_stride", "heads", "kv_heads", "d",
                                                 "dtype", "scale")), count, (C.c_int32 * 127)(*b))


CONFIGS = [
    (dict(n=-1), 1), (dict(n_seq=0), 1), (dict(n=1 << 31), 2), (dict(n_seq=1 << 31), 2), (dict(dtype=2), 2),
    (dict(d=0), 1), (dict(heads=0), 1), (dict(kv_heads=0), 1), (dict(d=12), 2), (dict(d=136, q_stride=1024, k_stride=512,
                                                                                      v_stride=512), 2),
    (dict(kv_heads=3, k_stride=96, v_stride=96), 1), (dict(heads=2048, q_stride=65536), 2), (dict(scale=0.0), 1),
    (dict(scale=-1.0), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1), (dict(q_stride=120), 1),
    (dict(q_stride=132), 1), (dict(k_stride=56), 1), (dict(v_stride=0), 1), (dict(q_stride=(1 << 23) + 8), 1),
    (dict(n_bounds=-1), 1), (dict(n_bounds=128), 1), (dict(bounds=(0, 1)), 1), (dict(bounds=(1, 1)), 1),
    (dict(bounds=(3, 2)), 1), (dict(bounds=(1, 4097)), 1),
]


@pytest.mark.parametrize("kw,status", CONFIGS)
def test_attention_configurations_refused(kw, status):
    n, c = C.c_size_t(), config(**kw)
    L = rece.lib()
    assert L.rece_attention_workspace_bytes(C.byref(c), C.byref(n)) == status
    assert L.rece_last_error().decode()
    assert L.rece_last_attention_workspace_bytes(C.byref(c), 100, C.byref(n)) == status
    assert L.rece_attention_forward(C.byref(c), None, P, P, P, P, None, None, 0, P) == status
    assert L.rece_last_attention(C.byref(c), None, 100, P, P, P, P, P, None, P, BIG, P) == status


def test_attention_without_configuration():
    n = C.c_size_t()
    assert rece.lib().rece_attention_workspace_bytes(None, C.byref(n)) == 1
    assert rece.lib().rece_attention_workspace_bytes(C.byref(config()), None) == 1
    assert rece.lib().rece_last_attention_workspace_bytes(C.byref(config()), 0, C.byref(n)) == 1
    assert rece.lib().rece_last_attention_workspace_bytes(C.byref(config()), 10, None) == 1


def test_attention_grids_beyond_the_device():
    n = C.c_size_t()
    c = config(n=1 << 30, n_seq=1)
    assert rece.lib().rece_attention_workspace_bytes(C.byref(c), C.byref(n)) == 2
    # a cache of as many rows is none
    assert rece.lib().rece_last_attention_workspace_bytes(C.byref(c), 100, C.byref(n)) == 0
    assert rece.lib().rece_last_attention_workspace_bytes(C.byref(config(n_seq=1 << 20)), 100, C.byref(n)) == 2
    c = config(heads=64, kv_heads=1, q_stride=64 * 32, k_stride=32, v_stride=32)
    assert rece.lib().rece_last_attention_workspace_bytes(C.byref(c), 100, C.byref(n)) == 2


def _fwd(**kw):
    a = dict(cfg=config(), q=P, k=P, v=P, offs=P, bias=None, ws=None, wsb=0, out=P)
    a.update(kw)
    return rece.lib().rece_attention_forward(C.byref(a["cfg"]), None, a["q"], a["k"], a["v"], a["offs"], a["bias"], a["ws"],
                                             a["wsb"], a["out"])


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(offs=None), 1), (dict(out=None), 1),
    (dict(q=C.c_void_p(24)), 1), (dict(k=C.c_void_p(8)), 1), (dict(out=C.c_void_p(40)), 1), (dict(offs=C.c_void_p(18)), 1),
    (dict(bias=C.c_void_p(18)), 1), (dict(ws=C.c_void_p(40), wsb=BIG), 1), (dict(ws=P, wsb=16), 3),
])
def test_attention_forward_refuses(kw, status):
    assert _fwd(**kw) == status


def test_attention_of_no_tokens_is_nothing():
    assert _fwd(cfg=config(n=0), q=None, k=None, v=None, offs=None, out=None) == 0


def _bwd(**kw):
    a = dict(cfg=config(bounds=(1, 2)), q=P, k=P, v=P, offs=P, bias=P, out=P, ws=P, wsb=BIG, dout=P, sq=128, sk=64, sv=64,
             dq=P, dk=P, dv=P, dbias=P)
    a.update(kw)
    return rece.lib().rece_attention_backward(C.byref(a["cfg"]), None, a["q"], a["k"], a["v"], a["offs"], a["bias"], a["out"],
                                              a["ws"], a["wsb"], a["dout"], a["sq"], a["sk"], a["sv"], a["dq"], a["dk"],
                                              a["dv"], a["dbias"])


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(offs=None), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(dout=None), 1), (dict(dq=None), 1),
    (dict(dk=None), 1), (dict(dv=None), 1), (dict(bias=None), 1), (dict(dbias=None), 1), (dict(sq=120), 1), (dict(sk=68), 1),
    (dict(sv=0), 1), (dict(sv=(1 << 23) + 8), 1), (dict(wsb=64), 3), (dict(dq=C.c_void_p(40)), 1),
    (dict(dout=C.c_void_p(40)), 1), (dict(dbias=C.c_void_p(18)), 1), (dict(ws=C.c_void_p(24)), 1),
])
def test_attention_backward_refuses(kw, status):
    assert _bwd(**kw) == status


def _last(**kw):
    a = dict(cfg=config(), max_len=5000, q=P, k=P, v=P, begin=P, length=P, bias=None, ws=P, wsb=BIG, out=P)
    a.update(kw)
    return rece.lib().rece_last_attention(C.byref(a["cfg"]), None, a["max_len"], a["q"], a["k"], a["v"], a["begin"],
                                          a["length"], a["bias"], a["ws"], a["wsb"], a["out"])


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(begin=None), 1), (dict(length=None), 1), (dict(out=None), 1),
    (dict(max_len=0), 1), (dict(q=C.c_void_p(8)), 1), (dict(begin=C.c_void_p(18)), 1), (dict(bias=C.c_void_p(18)), 1),
    (dict(ws=None), 3), (dict(wsb=100), 3),
])
def test_last_attention_refuses(kw, status):
    assert _last(**kw) == status


def _norm(name, **kw):
    a = dict(n=10, d=64, dtype=1, eps=1e-6, x=P, residual=P, weight=P, h=P, y=P, stat=P)
    a.update(kw)
    return getattr(rece.lib(), name)(None, a["n"], a["d"], a["dtype"], a["eps"], a["x"], a["residual"], a["weight"], a["h"],
                                     a["y"], a["stat"])


@pytest.mark.parametrize("name", ["rece_norm_forward", "rece_norm_forward_int8"])
@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(d=0), 1), (dict(d=12), 2), (dict(d=8200), 2), (dict(n=1 << 31), 2), (dict(dtype=3), 2),
    (dict(eps=-1.0), 1), (dict(eps=math.inf), 1), (dict(eps=math.nan), 1), (dict(x=None), 1), (dict(weight=None), 1),
    (dict(y=None), 1), (dict(x=C.c_void_p(8)), 1), (dict(residual=C.c_void_p(8)), 1), (dict(h=C.c_void_p(8)), 1),
    (dict(weight=C.c_void_p(8)), 1), (dict(stat=C.c_void_p(2)), 1),
])
def test_norm_refuses(name, kw, status):
    assert _norm(name, **kw) == status


def test_norm_takes_less():
    assert _norm("rece_norm_forward", n=0, x=None, weight=None, y=None) == 0
    assert _norm("rece_norm_forward_int8", stat=None) == 1
    n = C.c_size_t()
    assert rece.lib().rece_norm_workspace_bytes(10, 64, C.byref(n)) == 0 and n.value > 0
    assert rece.lib().rece_norm_workspace_bytes(10, 64, None) == 1 and rece.lib().rece_norm_workspace_bytes(10, 4, C.byref(n)) == 2


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), 1), (dict(h=None), 1), (dict(weight=None), 1), (dict(rstd=None), 1), (dict(ws=None), 1), (dict(dx=None), 1),
    (dict(dw=None), 1), (dict(wsb=8), 3), (dict(dy=C.c_void_p(8)), 1), (dict(dh=C.c_void_p(8)), 1), (dict(dw=C.c_void_p(2)), 1),
    (dict(dtype=9), 2), (dict(d=4), 2), (dict(n=-1), 1),
])
def test_norm_backward_refuses(kw, status):
    a = dict(n=10, d=64, dtype=1, dy=P, h=P, dh=None, weight=P, rstd=P, ws=P, wsb=BIG, dx=P, dw=P)
    a.update(kw)
    assert rece.lib().rece_norm_backward(None, *(a[k] for k in ("n", "d", "dtype", "dy", "h", "dh", "weight", "rstd", "ws", "wsb",
                                                                "dx", "dw"))) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(d=20), 2), (dict(dtype=2), 2), (dict(x=None), 1), (dict(x8=None), 1), (dict(scale=None), 1),
    (dict(x=C.c_void_p(8)), 1), (dict(x8=C.c_void_p(8)), 1), (dict(scale=C.c_void_p(2)), 1),
])
def test_quantize_rows_refuses(kw, status):
    a = dict(n=10, d=64, dtype=1, x=P, x8=P, scale=P)
    a.update(kw)
    assert rece.lib().rece_quantize_rows(None, *(a[k] for k in ("n", "d", "dtype", "x", "x8", "scale"))) == status


@pytest.mark.parametrize("kw,status", [
    (dict(s=-1), 1), (dict(C=0), 1), (dict(d=0), 1), (dict(d=24), 2), (dict(d=8208), 2), (dict(s=1 << 31), 2),
    (dict(C=1 << 31), 2), (dict(dtype=4), 2), (dict(x=None), 1), (dict(sx=None), 1), (dict(y=None), 1), (dict(sy=None), 1),
    (dict(out=None), 1), (dict(x=C.c_void_p(8)), 1), (dict(y=C.c_void_p(8)), 1), (dict(sx=C.c_void_p(2)), 1),
    (dict(out=C.c_void_p(1)), 1), (dict(out=C.c_void_p(2), dtype=0), 1), (dict(s=1 << 30, C=1 << 30, d=512), 2),
])
def test_scores_refuse(kw, status):
    a = dict(s=10, C=50, d=64, dtype=1, x=P, sx=P, y=P, sy=P, out=P)
    a.update(kw)
    assert rece.lib().rece_int8_scores(None, *(a[k] for k in ("s", "C", "d", "dtype", "x", "sx", "y", "sy", "out"))) == status


def test_binding_refuses():
    with pytest.raises(ValueError):
        rece.SequenceAttention(10, 2, 4, 32, dtype="f16")
    with pytest.raises(rece.ReceError):
        rece.SequenceAttention(10, 2, 4, 32, kv_heads=3)
    with pytest.raises(ValueError):
        rece.SequenceAttention(10, 2, 4, 32, bounds=list(range(1, 200)))
    with pytest.raises(ValueError):
        rece.ResidualNorm(10, 64, eps=-1.0)
    for bad in ((10, 5, 24), (10, 0, 32), (-1, 5, 32), (10, 5, 8208)):
        with pytest.raises(ValueError):
            rece.Int8Scores(*bad)
    op = rece.SequenceAttention(10, 2, 4, 32)
    t = torch.zeros(10, 4, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):       # not on a GPU
        op.forward(t, t, t, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        op.forward(t[0], t, t, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        rece.attention_qkv(torch.zeros(10, 64), torch.zeros(3, dtype=torch.int32), op)


@pytest.mark.parametrize("n_buckets,most", [(2, 2), (8, 20), (16, 128), (32, 128), (64, 4096), (126, 200)])
def test_log_buckets(n_buckets, most):
    bounds = rece.log_buckets(n_buckets, most)
    half = n_buckets // 2
    assert len(bounds) == n_buckets - 1 and bounds[:half] == list(range(1, half + 1))
    assert all(a < b for a, b in zip(bounds, bounds[1:])) and bounds[-1] <= max(most, n_buckets)
    for k, b in enumerate(bounds[half:], 1):
        exact = half * (most / half) ** (k / half)
        assert b >= exact - 1e-6 and (b - 1 < exact + 1e-6 or b == bounds[half + k - 2] + 1)


def test_log_buckets_refuses():
    for bad in ((3, 10), (0, 10), (32, 16), (32, 5000), (130, 4000)):
        with pytest.raises(ValueError):
            rece.log_buckets(*bad)
