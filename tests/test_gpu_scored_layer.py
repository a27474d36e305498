"""One training step of a routed layer through sigmoid scores with a bias and groups and through activations kept in 8 bits:
logits -> routing -> forward that saves codes -> layer output -> balance loss -> backward from the codes -> routing-weight and
logits' gradients -> update of weights and bias; against an fp64 model of the same step at the restored activations."""
import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
from oracle import checkpoint_oracle as co
from oracle import router_oracle as ro
from oracle import scored_oracle as so

from gpu_util import DEV, as_f64, log, rel_fro

pytestmark = pytest.mark.gpu

T, E, K, D, F = 413, 12, 3, 256, 136
COEF, RATE = 0.02, 1e-2
ROUTE = dict(renorm=True, scale=1.5, groups=4, top_groups=2, group_best=2)


def _bf(rng, *shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(DEV).bfloat16()


def _model(ref, X, W1, W2, G, H, Xr, keep):
    """fp64: layer output, and of the kept pairs dW1, dW2 at the restored rows H, Xr and the routing weights' gradient."""
    out, dW1, dW2, dw = np.zeros((T, D)), np.zeros_like(W1), np.zeros_like(W2), np.zeros((T, K))
    for j, (t, k) in enumerate(zip(ref["tok"], ref["slot"])):
        e, w = ref["idx"][t, k], ref["w"][t, k]
        g, u = np.split(X[t] @ W1[e], 2)
        y = (g * so.sigmoid(g) * u) @ W2[e]
        out[t] += w * y
        if keep[j]:
            dw[t, k] = G[t] @ y
            g, u = np.split(H[j], 2)
            sg, dphi = so.sigmoid(g), w * (W2[e] @ G[t])
            dW2[e] += np.outer(sg * g * u, w * G[t])
            dW1[e] += np.outer(Xr[t], np.concatenate([dphi * u * (sg + g * sg * (1 - sg)), dphi * sg * g]))
    return out, dW1, dW2, dw


@pytest.mark.parametrize("rho", [1.0, 0.5])
def test_training_step(rho):
    rng = np.random.default_rng(int(10 * rho) + 1)
    X, G = _bf(rng, T, D), _bf(rng, T, D)
    W1, W2 = _bf(rng, E, D, 2 * F, std=D ** -0.5), _bf(rng, E, F, D, std=F ** -0.5)
    logits = X.float() @ torch.from_numpy(rng.standard_normal((D, E)).astype(np.float32) * D ** -0.5).to(DEV)
    bias = torch.from_numpy((rng.standard_normal(E) * 0.05).astype(np.float32)).to(DEV)
    mask = torch.from_numpy((rng.random(T) < 0.9).astype(np.uint8)).to(DEV)
    off = [0, 130, 131, T]
    r = lr.Router(T=T, E=E, K=K, score="sigmoid", device=DEV, **ROUTE)

    log("routing")
    o = lr.route(r, logits, mask=mask, bias=bias)
    seg = o["seg_off"].cpu().numpy()
    N = int(seg[-1])
    quota = np.ceil(rho * np.diff(seg)).astype(np.int32)
    p = lr.Problem(E=E, T=T, K=K, D=D, F=F, swiglu=True, dtype=lr.BF16, seg_off=seg, quota=quota, device=DEV)
    log(f"expert forward over {N} pairs")
    X8 = lr.checkpoint(X)
    fw = lr.expert_forward_checkpoint(p, X, o["tok"], o["alpha"], W1, W2)
    y = lr.scatter(p, fw["Y"], o["tok"], o["slot"], n_rows=N)[:T]
    bal = lr.balance_loss(r, logits, o["idx"], coef=COEF, mask=mask, seq_off=off)
    log("expert backward")
    bw = lr.backward(p, G=G, H=fw["H"], X=X8, alpha=o["alpha"], tok=o["tok"], slot=o["slot"], W2=W2, W1=W1,
                     overlap_scatter=True)
    log("routing weights' and logits' gradients")
    da = lr.alpha_grad(p, G, fw["Y"], o["alpha"], o["pmap"], keep=bw["keep"])
    dx = lr.route_bwd(r, logits, o["idx"], dalpha=da, pmap=o["pmap"], balance=bal, mask=mask, seq_off=off)
    log("update")
    m1, m2 = W1.float(), W2.float()
    before = [as_f64(m1), as_f64(m2)]
    lr.AdamW([W1, W2], grads=[bw["dW1"], bw["dW2"]], masters=[m1, m2], bits=8, lr=1e-2).step()
    b1 = lr.bias_update(r, bias, o["counts"], RATE)
    torch.cuda.synchronize()

    L, M = as_f64(logits), mask.cpu().numpy()
    keep = bw["keep"].cpu().numpy() != 0
    ref = so.route(L, K, "sigmoid", as_f64(bias), mask=M, **ROUTE)
    assert np.array_equal(o["idx"].cpu().numpy(), ref["idx"]) and np.array_equal(seg, ref["seg_off"])
    H = co.values(fw["H"].q.cpu().numpy(), as_f64(fw["H"].scale))
    exact = np.concatenate([as_f64(X)[ref["tok"][seg[e]:seg[e + 1]]] @ before[0][e] for e in range(E)])
    # half a scale, which is 1.008 / 127 of a group's largest value at most, and the row's rounding to bf16
    half = np.repeat(as_f64(fw["H"].scale), 128, axis=2)[:, :, :F].reshape(N, 2 * F) / 2
    assert np.all(np.abs(H - exact) <= half + np.abs(exact) * 2.0 ** -8 + 1e-4)
    out, dW1, dW2, dw = _model(ref, as_f64(X), before[0], before[1], as_f64(G), H, as_f64(lr.restore(X8)), keep)
    assert int(keep.sum()) == int(quota.sum())
    # as for rows of the storage dtype: Y, PhiW and dH are rounded to bf16
    assert rel_fro(as_f64(y), out) <= 5e-3
    for got, want in ((bw["dW1"], dW1), (bw["dW2"], dW2)):
        assert rel_fro(as_f64(got), want) <= 5e-3
    b = so.balance(L, ref["idx"], COEF, "sigmoid", M, off)
    assert abs(float(bal["loss"]) - b["loss"]) <= b["loss_err"] + 2 ** -22 * b["loss"]
    assert rel_fro(as_f64(da), dw[ref["tok"], ref["slot"]]) <= 1e-2
    want, _ = so.sigmoid_bwd(L, ref["idx"], y=dw, counts=b["counts"], norm=b["norm"], mask=M, seq_off=off, renorm=True,
                             scale=1.5)
    assert rel_fro(as_f64(dx), want) <= 1e-2
    assert np.array_equal(b1.cpu().numpy(), so.bias_update(bias.cpu().numpy(), ref["counts"], RATE))
    zero = lambda a: np.zeros_like(a)  # noqa: E731
    for w, g, w0 in ((m1, bw["dW1"], before[0]), (m2, bw["dW2"], before[1])):
        (w1, _, _), (err, _, _) = ro.adamw(w0, as_f64(g), zero(w0), zero(w0), t=1, lr=1e-2, betas=(0.9, 0.999), eps=1e-8,
                                           weight_decay=0.01)
        assert np.all(np.abs(as_f64(w) - w1) <= err)
