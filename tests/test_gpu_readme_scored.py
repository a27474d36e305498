"""The README's training step with the lines of its second example in the place of the first one's: sigmoid scores, a bias and
groups, activations in 8 bits; run as they stand, against the oracle's choice and the backward from the restored rows."""
import re

import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr
from oracle import scored_oracle as so

from gpu_util import DEV, as_f64, log, rel_fro
from test_gpu_readme_step import README

pytestmark = pytest.mark.gpu


def _blocks():
    """(once, step) of both examples."""
    text = open(README, encoding="utf-8").read()
    code = [b for b in re.findall(r"```\n(.*?)```", text, re.S) if "lr.Router(" in b]
    assert len(code) == 2
    return [re.split(r"# every step.*\n", b) for b in code]


def _step(first, second):
    """The first example's step; lines whose result the second makes otherwise are the second's, and its others stand where
    they stand there."""
    name = lambda line: line.split(" = ")[0]  # noqa: E731
    lines, own = first.splitlines(), [x for x in second.splitlines() if x.strip()]
    have, out = {name(x) for x in lines if " = " in x}, []
    for line in lines:
        if " = " in line and name(line) in {name(x) for x in own}:
            while own and name(own[0]) != name(line):  # new ones before it
                assert name(own[0]) not in have
                out.append(own.pop(0))
            out.append(own.pop(0))
        else:
            out.append(line)
    return "\n".join(out + own)


def test_readme_step_in_8_bits():
    (once, step), (once2, step2) = _blocks()
    step = _step(step, step2)
    for call in ("lr.checkpoint(", "lr.expert_forward_checkpoint(", "H=f[\"H\"], X=X8", "lr.bias_update(", "bias=bias"):
        assert step.count(call) == 1, call
    T, E, K, D, F = 301, 16, 3, 128, 72
    rng = np.random.default_rng(37)

    def bf(*shape, std=1.0):
        return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(DEV).bfloat16()

    W1, W2 = bf(E, D, 2 * F, std=D ** -0.5), bf(E, F, D, std=F ** -0.5)
    env = {"lr": lr, "torch": torch, "T": T, "E": E, "K": K, "D": D, "F": F, "W1": W1, "W2": W2, "M1": W1.float(),
           "M2": W2.float(), "quotas": lambda seg_off: np.diff(seg_off).astype(np.int32)}

    def inputs():
        env.update(X=bf(T, D), G=bf(T, D), logits=torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV),
                   mask=torch.from_numpy(rng.random(T) < 0.9).to(DEV))

    log("what the README runs once")
    inputs()
    exec(once, env)
    exec(once2, env)
    for i in range(3):
        inputs()
        before, weights = env["bias"].cpu().numpy(), (W1.clone(), W2.clone())
        log(f"the README's step {i}, scores and 8 bits")
        exec(step, env)
        torch.cuda.synchronize()
        o, f, g, r, p = (env[k] for k in "ofgrp")
        ref = so.route(as_f64(env["logits"]), K, "sigmoid", before, r.groups, r.top_groups, r.group_best,
                       env["mask"].cpu().numpy(), given=o["idx"].cpu().numpy())
        assert np.array_equal(o["idx"].cpu().numpy(), ref["idx"]) and np.array_equal(o["counts"].cpu().numpy(), ref["counts"])
        assert np.array_equal(env["bias"].cpu().numpy(), so.bias_update(before, ref["counts"], 1e-3))
        assert (env["bias"].cpu().numpy() != before).any()
        H = lr.restore(f["H"])
        gate, up = H.float().split(F, dim=1)
        plain = lr.backward(p, G=env["G"], Phi=(gate * torch.sigmoid(gate) * up).bfloat16(), H=H, X=lr.restore(env["X8"]),
                            alpha=o["alpha"], tok=o["tok"], slot=o["slot"], W2=weights[1], W1=weights[0])
        # six roundings to bf16 lie between the two (gate, up and Phi of the one, PhiW, dH and dIn of both), each half a step
        # of 2^-8 at most, under 2e-3 rms: 5e-3 together
        for k in ("dW1", "dW2", "out"):
            assert rel_fro(as_f64(g[k]), as_f64(plain[k])) <= 1e-2, k
        assert env["dlogits"].shape == (T, E) and env["y"].shape == (T, D) and float(env["b"]["loss"]) > 0
        assert not torch.equal(W1, weights[0]) and not torch.equal(W2, weights[1])
