"""Activation checkpoints in 8 bits without a GPU: the definition, refusals of the C calls and of the binding."""
import ctypes
import types

import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
from load_recalibrated_expert_amd import _lib
from oracle import checkpoint_oracle as co
import oracle

from test_router_binding_cpu import Stream, Tensor, gpu  # noqa: F401

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1001)


# ------------------------------------------------------------------------------- the definition

def test_codes_by_hand():
    x = np.zeros((1, 128))
    x[0, :6] = [127.0, -127.0, 0.5, 1.5, -2.5, 0.49]  # the scale is 1: ties go to even
    q, s = co.checkpoint(x, 1)
    assert s[0, 0, 0] == 1.0 and q[0, :6].tolist() == [127, -127, 0, 2, -2, 0]
    x[0, 0] = 127.25  # no longer: the next bf16 number above 1 is 1 + 2^-7
    assert co.checkpoint(x, 1)[1][0, 0, 0] == 1 + 2.0 ** -7
    q, s = co.checkpoint(np.zeros((1, 8)), 1)
    assert s[0, 0, 0] == 2.0 ** -126 and not q.any()


@pytest.mark.parametrize("parts,width", [(1, 8), (1, 136), (2, 768), (3, 264)])
def test_values_are_within_half_a_scale(parts, width):
    rng = np.random.default_rng(width)
    x = (rng.standard_normal((50, parts * width)) * np.exp(rng.standard_normal((50, 1)) * 20)).astype(np.float32)
    q, s = co.checkpoint(x, parts)
    assert np.abs(q).max() <= 127 and s.shape == (50, parts, co.groups(width))
    half = np.repeat(s, co.GROUP, axis=2)[:, :, :width].reshape(50, -1) / 2
    assert np.all(np.abs(co.values(q, s) - x) <= half)
    # the scale is a bf16 number, large enough, and the one before is not
    b = torch.from_numpy(s).bfloat16()
    assert np.array_equal(b.double().numpy(), s)
    before = (b.view(torch.int16) - 1).view(torch.bfloat16).double().numpy()
    amax = np.abs(co._split(x, parts)).max(3)
    assert np.all(127 * s >= amax) and np.all((127 * before < amax) | (s == 2.0 ** -126))


def test_a_group_with_a_bad_value_is_nan():
    x = np.ones((2, 256))
    x[0, 130], x[1, 5] = np.inf, np.nan
    q, s = co.checkpoint(x, 1)
    v = co.values(q, s)
    assert np.isnan(v[0, 128:]).all() and np.isnan(v[1, :128]).all()
    assert np.abs(v[0, :128] - 1).max() < 0.01 and np.abs(v[1, 128:] - 1).max() < 0.01


def test_activation_backward_against_differences():
    """dH from restored rows is the derivative of the output there: L = sum alpha <g, phi(h) W2>."""
    rng = np.random.default_rng(4)
    n, F, D, h = 3, 5, 4, 1e-6
    H, g, W2, a = rng.standard_normal((n, 2 * F)) * 2, rng.standard_normal((n, D)), rng.standard_normal((F, D)), rng.random(n)
    q, s = co.checkpoint(np.pad(H.reshape(n, 2, F), ((0, 0), (0, 0), (0, 3))).reshape(n, 16), 2)
    V = co.values(q, s).reshape(n, 2, 8)[:, :, :F].reshape(n, 2 * F)
    P = co.phi(V, True)[0]
    row_off = np.array([0, n])
    dW1, dW2, dH, dX = oracle.swiglu_expert_backward(row_off, a[:, None] * g, P, rng.standard_normal((n, D)), V,
                                                     rng.standard_normal((1, D, 2 * F)), W2[None])
    loss = lambda v: (a[:, None] * g * (co.phi(v, True)[0] @ W2)).sum()  # noqa: E731
    for i in range(n):
        for c in range(2 * F):
            up, down = V.copy(), V.copy()
            up[i, c] += h
            down[i, c] -= h
            # cancellation of order 2^-52 / h and a third derivative of order 10 times h^2
            assert abs((loss(up) - loss(down)) / (2 * h) - dH[i, c]) < 1e-8
    assert np.allclose(dW2[0], (a[:, None] * P).T @ g, rtol=1e-13)


# ------------------------------------------------------------------------------- refusals

def test_checkpoint_and_restore_refusals():
    lib = _lib.load()

    def both(n=4, parts=2, width=16, dtype=_lib.BF16, rows=FAKE, q=FAKE, scale=FAKE):
        a = lib.lrmoe_checkpoint(n, parts, width, dtype, rows, q, scale, None)
        b = lib.lrmoe_restore(n, parts, width, q, scale, dtype, rows, None)
        assert a == b
        return a

    for kw in (dict(n=-1), dict(parts=0), dict(width=0), dict(width=-8), dict(rows=None), dict(q=None),
               dict(scale=None), dict(rows=ctypes.c_void_p(0x1008)), dict(q=ctypes.c_void_p(0x1008)), dict(scale=ODD)):
        assert both(**kw) == _lib.ERR_INVALID_ARG, kw
    for kw in (dict(width=12), dict(dtype=2), dict(n=2 ** 30, parts=1, width=128), dict(n=2 ** 22, width=2 ** 14),
               dict(n=2 ** 62), dict(parts=2 ** 30, n=2 ** 39)):
        assert both(**kw) == _lib.ERR_UNSUPPORTED, kw
    assert both(n=0, rows=None, q=None, scale=None) == _lib.OK


def _problem(swiglu=True, dtype=_lib.BF16, D=64, F=32):
    return _lib.make_problem_struct(2, 6, 2, D, F, swiglu, dtype, [0, 5, 9], [5, 4])


def test_step_refusals():
    lib = _lib.load()
    p, keep = _problem()
    bad, keep2 = _problem(F=30)
    lin, keep3 = _problem(swiglu=False)
    n = ctypes.c_size_t(0)
    lib.lrmoe_workspace_size(ctypes.byref(p), 0, ctypes.byref(n))

    def score(prob=p, ws=FAKE, nb=n.value, **kw):
        a = dict(G=FAKE, q=FAKE, scale=FAKE, alpha=FAKE, tok=FAKE, R=FAKE)
        a.update(kw)
        return lib.lrmoe_score_checkpoint(ctypes.byref(prob), *a.values(), ws, nb, None)

    def compact(prob=p, **kw):
        a = dict(sel=FAKE, q=FAKE, scale=FAKE, alpha=FAKE, PhiW=FAKE)
        a.update(kw)
        return lib.lrmoe_compact_checkpoint(ctypes.byref(prob), *a.values(), None)

    def forward(prob=p, **kw):
        a = dict(seg=FAKE, X=FAKE, tok=FAKE, alpha=FAKE, W1=FAKE, W2=FAKE, q=FAKE, scale=FAKE, Phi=FAKE, Y=FAKE)
        a.update(kw)
        return lib.lrmoe_expert_forward_checkpoint(ctypes.byref(prob), *a.values(), None)

    def gemm(prob=p, acc=0, ws=FAKE, nb=n.value, **kw):
        a = dict(off=FAKE, G=FAKE, alpha=FAKE, sel=FAKE, ctok=FAKE, PhiW=FAKE, X=FAKE, q=FAKE, scale=FAKE, W2=FAKE,
                 W1=FAKE, dW2=FAKE, dW1=FAKE, dH=FAKE, dIn=FAKE)
        a.update(kw)
        return lib.lrmoe_grouped_gemm_bwd_checkpoint(ctypes.byref(prob), *a.values(), acc, ws, nb, None, None)

    for call, names in ((score, ("G", "q", "scale", "alpha", "tok", "R")),
                        (compact, ("sel", "q", "scale", "alpha", "PhiW")),
                        (forward, ("seg", "X", "tok", "alpha", "W1", "W2", "q", "scale", "Phi", "Y")),
                        (gemm, ("off", "G", "alpha", "sel", "ctok", "PhiW", "X", "q", "scale", "W2", "W1", "dW2", "dW1",
                                "dH", "dIn"))):
        for name in names:
            assert call(**{name: None}) == _lib.ERR_INVALID_ARG, (call, name)
        assert call(scale=ODD) == _lib.ERR_INVALID_ARG
        assert call(q=ctypes.c_void_p(0x1008)) == _lib.ERR_INVALID_ARG
        assert call(prob=bad) == _lib.ERR_UNSUPPORTED
    assert score(ws=None) == score(nb=1) == gemm(ws=None) == gemm(nb=1) == _lib.ERR_WORKSPACE
    assert gemm(acc=2) == _lib.ERR_INVALID_ARG
    assert gemm(prob=lin) == forward(prob=lin) == _lib.ERR_UNSUPPORTED


def test_python_refusals(gpu):  # noqa: F811
    i8, bf, f32 = torch.int8, torch.bfloat16, torch.float32
    good = lr.Checkpoint(Tensor((9, 64), i8, 0), Tensor((9, 2, 1), bf, 0))
    for q, s in ((Tensor((9, 64), torch.uint8, 0), Tensor((9, 2, 1), bf, 0)),
                 (Tensor((9, 64), i8, 0), Tensor((9, 2, 1), f32, 0)), (Tensor((9, 64), i8, 0), Tensor((9, 2), bf, 0)),
                 (Tensor((9, 64), i8, 0), Tensor((8, 2, 1), bf, 0)), (Tensor((9, 64), i8, 0), Tensor((9, 3, 1), bf, 0)),
                 (Tensor((9, 640), i8, 0), Tensor((9, 2, 2), bf, 0)), (Tensor((9, 64), i8, 0), Tensor((9, 2, 1), bf, 1)),
                 (Tensor((576,), i8, 0), Tensor((9, 2, 1), bf, 0))):
        with pytest.raises(ValueError):
            lr.Checkpoint(q, s)
    for rows, kw in ((Tensor((9, 64), torch.float16, 0), {}), (Tensor((9, 64), bf, 1), {}), (Tensor((9, 60), bf, 0), {}),
                     (Tensor((9, 64), bf, 0), dict(parts=3)), (Tensor((9, 64), bf, 0), dict(parts=0)),
                     (Tensor((9, 64), bf, 0), dict(parts=16)), (Tensor((576,), bf, 0), {}),
                     (Tensor((9, 64), bf, 0), dict(out=good)), (Tensor((10, 64), bf, 0), dict(parts=2, out=good)),
                     (Tensor((9, 64), bf, 0), dict(parts=2, stream=Stream(1, 7001)))):
        with pytest.raises(ValueError):
            lr.checkpoint(rows, **kw)
    for kw in (dict(dtype=torch.float16), dict(out=Tensor((9, 32), bf, 0)), dict(out=Tensor((9, 64), bf, 1)),
               dict(stream=Stream(1, 7001))):
        with pytest.raises(ValueError):
            lr.restore(good, **kw)
    p = types.SimpleNamespace(N=9, T=8, K=2, D=8, F=32, K_tot=5, swiglu=True, torch_dtype=bf, device="cuda:0",
                              c=_lib.CProblem(), workspace=lambda mode=0: Tensor((512,), torch.uint8, 0))
    lin = types.SimpleNamespace(**{**vars(p), "swiglu": False})
    few = lr.Checkpoint(Tensor((8, 64), i8, 0), Tensor((8, 2, 1), bf, 0))
    other = lr.Checkpoint(Tensor((9, 64), i8, 1), Tensor((9, 2, 1), bf, 1))
    one = lr.Checkpoint(Tensor((9, 64), i8, 0), Tensor((9, 1, 1), bf, 0))
    t = Tensor((9,), f32, 0)
    for H, prob in ((few, p), (other, p), (one, p), (good, lin)):
        with pytest.raises(ValueError):
            lr.score_checkpoint(prob, t, H, t, t)
        with pytest.raises(ValueError):
            lr.compact_checkpoint(prob, t, H, t)
        with pytest.raises(ValueError):
            lr.grouped_gemm_bwd_checkpoint(prob, t, t, t, t, t, t, t, H, t)
    with pytest.raises(ValueError):
        lr.expert_forward_checkpoint(p, t, t, t, t, t, out={"H": few, "Phi": t, "Y": t})
    common = dict(G=t, alpha=t, tok=t, slot=t, W2=t, stream=Stream(0, 7000))
    x8 = lr.Checkpoint(Tensor((8, 8), i8, 0), Tensor((8, 1, 1), bf, 0))
    for kw in (dict(H=good, Phi=t), dict(), dict(Phi=one), dict(H=good, mode=lr.COMPACT_ZERO_MASKED),
               dict(H=good, packed_dlt=True), dict(H=t, Phi=t, X=x8, packed_dlt=True),
               dict(H=good, X=lr.Checkpoint(Tensor((7, 8), i8, 0), Tensor((7, 1, 1), bf, 0)))):
        with pytest.raises(ValueError):
            lr.backward(p, **common, **kw)
    with pytest.raises(ValueError):
        lr.backward(lin, **common, H=good)
    with pytest.raises(ValueError):
        lr.backward(lin, **common, Phi=lr.Checkpoint(Tensor((9, 32), i8, 0), Tensor((9, 1, 1), bf, 0)), X=x8)
    assert gpu.lib.launched == []


def test_gemm_is_for_gate_and_up(gpu):  # noqa: F811
    bf = torch.bfloat16
    lin = types.SimpleNamespace(N=9, T=8, K=2, D=8, F=32, K_tot=5, swiglu=False, torch_dtype=bf, device="cuda:0",
                                c=_lib.CProblem(), workspace=lambda mode=0: Tensor((512,), torch.uint8, 0))
    phi, t = lr.Checkpoint(Tensor((9, 32), torch.int8, 0), Tensor((9, 1, 1), bf, 0)), Tensor((9,), torch.float32, 0)
    with pytest.raises(ValueError):
        lr.grouped_gemm_bwd_checkpoint(lin, t, t, t, t, t, t, t, phi, t, out=dict(dW2=t, dIn=t))
    assert gpu.lib.launched == []
