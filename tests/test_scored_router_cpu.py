"""Routing by scores without a GPU: refusals (host checks before any launch, and the binding's), and the fp64
definitions against differences and counts of their own."""
import ctypes

import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
from load_recalibrated_expert_amd import _lib
from oracle import router_oracle as ro
from oracle import scored_oracle as so

from test_router_binding_cpu import Stream, Tensor, gpu  # noqa: F401

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1002)


def _router(**kw):
    d = dict(T=10, E=16, K=4, first=0, local=16, dtype=_lib.F32, renorm=0, reserved=0, scale=1.0)
    d.update(kw)
    return _lib.CRouter(**d)


def _scoring(**kw):
    d = dict(score=1, groups=4, top_groups=2, group_best=2)
    d.update(kw)
    return _lib.CScoring(**d)


def _size(r):
    n = ctypes.c_size_t(0)
    assert _lib.load().lrmoe_router_workspace_size(ctypes.byref(r), 3, ctypes.byref(n)) == _lib.OK
    return n.value


@pytest.mark.parametrize("kw,expect", [
    ({}, _lib.OK), (dict(groups=1, top_groups=1), _lib.OK), (dict(groups=16, top_groups=4, group_best=1), _lib.OK),
    (dict(score=0), _lib.OK), (dict(groups=4, top_groups=1), _lib.OK),
    (dict(score=2), _lib.ERR_INVALID_ARG), (dict(score=-1), _lib.ERR_INVALID_ARG),
    (dict(groups=0), _lib.ERR_INVALID_ARG), (dict(groups=-4), _lib.ERR_INVALID_ARG),
    (dict(groups=3), _lib.ERR_INVALID_ARG), (dict(groups=32), _lib.ERR_INVALID_ARG),
    (dict(top_groups=0), _lib.ERR_INVALID_ARG), (dict(top_groups=5), _lib.ERR_INVALID_ARG),
    (dict(group_best=0), _lib.ERR_INVALID_ARG), (dict(group_best=3), _lib.ERR_INVALID_ARG),
    (dict(groups=16, top_groups=3), _lib.ERR_INVALID_ARG),  # three experts for four slots
])
def test_scoring_checks(kw, expect):
    c = _scoring(**kw)
    assert _lib.load().lrmoe_scoring_check(ctypes.byref(_router()), ctypes.byref(c)) == expect


def test_more_groups_than_marks_are_refused():
    lib = _lib.load()
    for E, groups, expect in ((128, 64, _lib.OK), (128, 128, _lib.ERR_UNSUPPORTED)):
        r, c = _router(E=E, local=E), _scoring(groups=groups, top_groups=groups)
        assert lib.lrmoe_scoring_check(ctypes.byref(r), ctypes.byref(c)) == expect
    assert lib.lrmoe_scoring_check(None, ctypes.byref(_scoring())) == _lib.ERR_INVALID_ARG
    assert lib.lrmoe_scoring_check(ctypes.byref(_router()), None) == _lib.ERR_INVALID_ARG


def test_route_refusals():
    lib, r, c = _lib.load(), _router(), _scoring()
    n = _size(r)

    def call(ptrs=None, ws=FAKE, nb=n, router=r, scoring=c):
        p = {k: FAKE for k in ("logits", "bias", "idx", "w", "counts", "seg_off", "tok", "slot", "alpha", "pmap")}
        p.update(ptrs or {})
        return lib.lrmoe_route_scored(ctypes.byref(router), ctypes.byref(scoring), p["logits"], p["bias"], None,
                                      p["idx"], p["w"], p["counts"], p["seg_off"], p["tok"], p["slot"], p["alpha"],
                                      p["pmap"], ws, nb, None)

    for name in ("logits", "idx", "w", "counts", "seg_off", "tok", "slot", "alpha", "pmap"):
        assert call({name: None}) == _lib.ERR_INVALID_ARG, name
    assert call({"logits": ODD}) == call({"bias": ODD}) == _lib.ERR_INVALID_ARG
    assert call(ws=None) == call(nb=0) == _lib.ERR_WORKSPACE
    assert call(router=_router(K=0)) == call(scoring=_scoring(groups=5)) == _lib.ERR_INVALID_ARG


def test_balance_and_gradient_refusals():
    lib, r, c = _lib.load(), _router(), _scoring()
    n = _size(r)

    def balance(logits=FAKE, idx=FAKE, off=FAKE, n_seq=3, coef=0.1, counts=FAKE, ws=FAKE, nb=n, scoring=c):
        return lib.lrmoe_balance_loss_scored(ctypes.byref(r), ctypes.byref(scoring), logits, None, idx, off, n_seq, coef,
                                             counts, FAKE, FAKE, FAKE, ws, nb, None)

    def grad(logits=FAKE, idx=FAKE, dalpha=FAKE, pmap=FAKE, n_pairs=5, off=FAKE, n_seq=2, counts=FAKE, norm=FAKE,
             out=FAKE, scoring=c):
        return lib.lrmoe_route_bwd_scored(ctypes.byref(r), ctypes.byref(scoring), logits, None, idx, dalpha, pmap,
                                          n_pairs, off, n_seq, counts, norm, None, out, None)

    bad = dict(scoring=_scoring(score=7))
    for kw in (dict(logits=None), dict(logits=ODD), dict(idx=None), dict(off=None), dict(n_seq=0),
               dict(coef=float("inf")), dict(counts=None), bad):
        assert balance(**kw) == _lib.ERR_INVALID_ARG, kw
    assert balance(ws=None) == balance(nb=16) == _lib.ERR_WORKSPACE
    for kw in (dict(logits=None), dict(out=None), dict(out=ODD), dict(idx=None), dict(n_pairs=-1), dict(counts=None),
               dict(off=None), dict(n_seq=0), bad):
        assert grad(**kw) == _lib.ERR_INVALID_ARG, kw


def test_bias_update_refusals():
    lib, r = _lib.load(), _router()

    def call(counts=FAKE, rate=1e-3, bias=FAKE, out=FAKE, router=r):
        return lib.lrmoe_bias_update(ctypes.byref(router), counts, rate, bias, out, None)

    for kw in (dict(counts=None), dict(bias=None), dict(out=None), dict(counts=ODD), dict(bias=ODD), dict(out=ODD),
               dict(rate=float("nan")), dict(rate=float("inf")), dict(router=_router(E=0))):
        assert call(**kw) == _lib.ERR_INVALID_ARG, kw


def test_python_refusals():
    new = lambda **kw: lr.Router(T=8, E=12, K=2, device="cuda:0", **kw)  # noqa: E731
    with pytest.raises(ValueError):
        new(score="relu")
    for kw in (dict(groups=5), dict(groups=3, top_groups=4), dict(group_best=3), dict(top_groups=2),
               dict(score="sigmoid", groups=12, top_groups=1)):
        with pytest.raises(lr.LrmoeError):
            new(**kw)


def test_binding_checks_the_bias_and_dispatches(gpu):  # noqa: F811
    x, f32 = Tensor((8, 12), torch.float32, 0), torch.float32
    plain = lr.Router(T=8, E=12, K=2, device="cuda:0")
    sig = lr.Router(T=8, E=12, K=2, score="sigmoid", device="cuda:0")
    gpu.lib.launched.clear()
    idx = Tensor((8, 2), torch.int32, 0)
    bal = {"counts": Tensor((1, 12), torch.int32, 0), "norm": Tensor((1,), f32, 0)}
    for bias in (Tensor((11,), f32, 0), Tensor((12,), torch.float64, 0), Tensor((12,), f32, 1), Tensor((1, 12), f32, 0)):
        for r in (plain, sig):
            with pytest.raises(ValueError):
                lr.route(r, x, bias=bias)
        with pytest.raises(ValueError):
            lr.bias_update(sig, bias, Tensor((12,), torch.int32, 0), 1e-3)
    for counts in (Tensor((12,), torch.int64, 0), Tensor((11,), torch.int32, 0), Tensor((12,), torch.int32, -1)):
        with pytest.raises(ValueError):
            lr.bias_update(sig, Tensor((12,), f32, 0), counts, 1e-3)
    bias, counts = Tensor((12,), f32, 0), Tensor((12,), torch.int32, 0)
    for call in (lambda s: lr.route(sig, x, stream=s), lambda s: lr.bias_update(sig, bias, counts, 1e-3, stream=s)):
        with pytest.raises(ValueError):
            call(Stream(1, 7001))
    assert gpu.lib.launched == []
    lr.route(plain, x)
    lr.route(plain, x, bias=bias)
    lr.route(sig, x)
    lr.balance_loss(sig, x, idx)
    lr.route_bwd(sig, x, idx, balance=bal)
    lr.bias_update(sig, bias, counts, 1e-3)
    assert gpu.lib.launched == ["lrmoe_route", "lrmoe_route_scored", "lrmoe_route_scored", "lrmoe_balance_loss_scored",
                                "lrmoe_route_bwd_scored", "lrmoe_bias_update"]


# ------------------------------------------------------------------------------- the definitions

def _weights(x, idx, renorm, scale):
    xk = np.take_along_axis(x, np.maximum(idx, 0), 1)
    s = np.where(idx >= 0, so.sigmoid(xk), 0)
    return scale * (s / s.sum(1, keepdims=True) if renorm else s)


@pytest.mark.parametrize("renorm", [False, True])
def test_weight_gradient_against_differences(renorm):
    rng = np.random.default_rng(1)
    T, E, K, h = 6, 9, 3, 1e-6
    x, y = rng.standard_normal((T, E)) * 2, rng.standard_normal((T, K))
    x[2, 4] = -np.inf
    idx = so.route(x, K, "sigmoid", bias=rng.standard_normal(E))["idx"]
    dx, _ = so.sigmoid_bwd(x, idx, y=y, renorm=renorm, scale=1.5)
    for t in range(T):
        for e in range(E):
            if x[t, e] == -np.inf:
                assert dx[t, e] == 0
                continue
            up, down = x.copy(), x.copy()
            up[t, e] += h
            down[t, e] -= h
            d = ((_weights(up, idx, renorm, 1.5) - _weights(down, idx, renorm, 1.5)) * y).sum() / (2 * h)
            # differences: cancellation of order 2^-52 / h and a third derivative of order 1 times h^2
            assert abs(d - dx[t, e]) < 1e-8


def test_balance_gradient_against_differences():
    rng = np.random.default_rng(2)
    T, E, K, h = 12, 7, 2, 1e-6
    x = rng.standard_normal((T, E))
    off = [0, 5, 5, 12]
    idx = so.route(x, K, "sigmoid")["idx"]
    b = so.balance(x, idx, 0.5, "sigmoid", seq_off=off)
    dx, _ = so.sigmoid_bwd(x, idx, counts=b["counts"], norm=b["norm"], gloss=0.7, seq_off=off)
    for t in range(T):
        for e in range(E):
            up, down = x.copy(), x.copy()
            up[t, e] += h
            down[t, e] -= h
            d = 0.7 * (so.balance(up, idx, 0.5, "sigmoid", seq_off=off)["loss"] -
                       so.balance(down, idx, 0.5, "sigmoid", seq_off=off)["loss"]) / (2 * h)
            assert abs(d - dx[t, e]) < 1e-8


def test_softmax_without_bias_and_groups_is_the_plain_router():
    x = np.random.default_rng(3).standard_normal((40, 24))
    x[5, :20], x[6] = np.nan, -np.inf
    a, b = ro.route(x, 6, renorm=True, first=3, local=9), so.route(x, 6, "softmax", renorm=True, first=3, local=9)
    for k in ("idx", "counts", "seg_off", "tok", "slot", "pmap"):
        assert np.array_equal(a[k], b[k]), k
    assert np.allclose(a["w"], b["w"], rtol=1e-14, atol=0)


def test_groups_by_hand():
    x = np.log(np.array([[0.9, 0.1, 0.6, 0.6, 0.7, 0.65]]) / (1 - np.array([[0.9, 0.1, 0.6, 0.6, 0.7, 0.65]])))
    pick = lambda **kw: so.route(x, 2, "sigmoid", groups=3, **kw)["idx"][0].tolist()  # noqa: E731
    assert pick(top_groups=1, group_best=1) == [0, 1]
    assert pick(top_groups=1, group_best=2) == [4, 5]  # 1.35 against 1.0 and 1.2
    assert pick(top_groups=2, group_best=2) == [4, 5]
    assert pick(top_groups=2, group_best=1) == [0, 4]
    assert pick(top_groups=1, group_best=2, bias=[0, 0, 0.2, 0, 0, 0]) == [2, 3]
    assert pick(top_groups=1, group_best=1, bias=[-np.inf, 0, 0, 0, 0, 0]) == [4, 5]


def test_bias_steps():
    assert so.bias_update([0.5, 0.5, 0.5], [1, 2, 3], 0.25).tolist() == [0.75, 0.5, 0.25]
    assert so.bias_update([0.5, -1], [2, 2], 0.25).tolist() == [0.5, -1]
