"""One training step of a routed layer with every operator as a program uses them together: logits ->
routing and pair lists -> expert forward -> layer output -> balance loss -> score, selection and
the expert backward on the retained pairs -> routing-weight gradient -> logits' gradient -> AdamW on
the experts' weights and the router's; against an fp64 model of the same step."""
import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
from oracle import router_oracle as ro

from gpu_util import DEV, as_f64, log, rel_fro

pytestmark = pytest.mark.gpu

T, E, K, D, F = 413, 6, 3, 256, 136
COEF = 0.02


def _bf(rng, *shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(DEV).bfloat16()


def _model(X, W1, W2, logits, mask, G, keep_rows=None):
    """fp64: layer output, dW1, dW2 over the kept pairs, gradient of the routing weights by slot."""
    r = ro.route(logits, K, mask, renorm=True, scale=1.5)
    out = np.zeros((T, D))
    dW1, dW2 = np.zeros_like(W1), np.zeros_like(W2)
    dw = np.zeros((T, K))
    for j, (t, k) in enumerate(zip(r["tok"], r["slot"])):
        e = r["idx"][t, k]
        h = X[t] @ W1[e]
        g, u = h[:F], h[F:]
        sg = 1 / (1 + np.exp(-g))
        phi = sg * g * u
        y = phi @ W2[e]
        out[t] += r["w"][t, k] * y
        if keep_rows is None or keep_rows[j]:
            dw[t, k] = G[t] @ y
            dphi = r["w"][t, k] * (W2[e] @ G[t])
            dh = np.concatenate([dphi * u * (sg + g * sg * (1 - sg)), dphi * sg * g])
            dW2[e] += np.outer(phi, r["w"][t, k] * G[t])
            dW1[e] += np.outer(X[t], dh)
    return r, out, dW1, dW2, dw


@pytest.mark.parametrize("rho", [1.0, 0.5])
def test_training_step(rho):
    rng = np.random.default_rng(int(10 * rho))
    X, G = _bf(rng, T, D), _bf(rng, T, D)
    W1, W2 = _bf(rng, E, D, 2 * F, std=D ** -0.5), _bf(rng, E, F, D, std=F ** -0.5)
    Wr = torch.from_numpy(rng.standard_normal((D, E)).astype(np.float32) * D ** -0.5).to(DEV)
    mask = torch.from_numpy((rng.random(T) < 0.9).astype(np.uint8)).to(DEV)
    off = [0, 130, 131, T]
    logits = X.float() @ Wr
    r = lr.Router(T=T, E=E, K=K, renorm=True, scale=1.5, device=DEV)

    log("routing")
    o = lr.route(r, logits, mask=mask)
    seg = o["seg_off"].cpu().numpy()
    N = int(seg[-1])
    quota = np.ceil(rho * np.diff(seg)).astype(np.int32)
    p = lr.Problem(E=E, T=T, K=K, D=D, F=F, swiglu=True, dtype=lr.BF16, seg_off=seg, quota=quota, device=DEV)
    log(f"expert forward over {N} pairs")
    fw = lr.expert_forward(p, X, o["tok"], o["alpha"], W1, W2)
    y = lr.scatter(p, fw["Y"], o["tok"], o["slot"], n_rows=N)[:T]
    log("balance loss")
    bal = lr.balance_loss(r, logits, o["idx"], coef=COEF, mask=mask, seq_off=off)
    log("expert backward")
    bw = lr.backward(p, G=G, Phi=fw["Phi"], alpha=o["alpha"], tok=o["tok"], slot=o["slot"], W2=W2, X=X, H=fw["H"],
                     W1=W1, overlap_scatter=True)
    log("routing weights' and logits' gradients")
    da = lr.alpha_grad(p, G, fw["Y"], o["alpha"], o["pmap"], keep=bw["keep"])
    dx = lr.route_bwd(r, logits, o["idx"], dalpha=da, pmap=o["pmap"], balance=bal, mask=mask, seq_off=off)
    dWr = X.float().t() @ dx
    log("update")
    m1, m2 = W1.float(), W2.float()
    before = [as_f64(m1), as_f64(m2), as_f64(Wr)]
    hyper = dict(lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
    experts = lr.AdamW([W1, W2], grads=[bw["dW1"], bw["dW2"]], masters=[m1, m2], bits=8, **hyper)
    router = lr.AdamW([Wr], grads=[dWr], **hyper)
    experts.step()
    router.step()
    torch.cuda.synchronize()

    L, M = as_f64(logits), mask.cpu().numpy()
    keep = bw["keep"].cpu().numpy() != 0
    ref, out, dW1, dW2, dw = _model(as_f64(X), before[0], before[1], L, M, as_f64(G), keep)
    assert np.array_equal(o["idx"].cpu().numpy(), ref["idx"]) and np.array_equal(seg, ref["seg_off"])
    assert int(keep.sum()) == int(quota.sum())
    # Y, H and Phi are rounded to bf16 (2^-9 rms each), sums of up to K of them: the forward suite's bound
    assert rel_fro(as_f64(y), out) <= 5e-3
    for got, want in ((bw["dW1"], dW1), (bw["dW2"], dW2)):
        assert rel_fro(as_f64(got), want) <= 1e-2  # the backward suite's 5e-3 and the forward's
    b = ro.balance(L, ref["idx"], COEF, M, off)
    assert abs(float(bal["loss"]) - b["loss"]) <= b["loss_err"] + 2 ** -22 * b["loss"]
    # the rounded rows reach dw as 2^-9 of the terms of a sum of D products, whose signs differ
    assert rel_fro(as_f64(da), dw[ref["tok"], ref["slot"]]) <= 1e-2
    want, _ = ro.route_bwd(L, ref["idx"], y=dw, counts=b["counts"], norm=b["norm"], mask=M, seq_off=off, renorm=True,
                           scale=1.5)
    assert rel_fro(as_f64(dx), want) <= 1e-2
    zero = lambda a: np.zeros_like(a)  # noqa: E731
    for w, g, w0 in ((m1, bw["dW1"], before[0]), (m2, bw["dW2"], before[1]), (Wr, dWr, before[2])):
        (w1, _, _), (err, _, _) = ro.adamw(w0, as_f64(g), zero(w0), zero(w0), t=1, **hyper)
        assert np.all(np.abs(as_f64(w) - w1) <= err)
    assert torch.equal(W1, m1.bfloat16()) and torch.equal(W2, m2.bfloat16())
