"""The training step that the README shows, run as it stands: every step's update takes that step's gradients."""
import os
import re

import numpy as np
import pytest
import torch

import load_recalibrated_expert_amd as lr

from gpu_util import DEV, log

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def _example():
    """(what is run once, what is run at every step)"""
    text = open(README, encoding="utf-8").read()
    code = next(b for b in re.findall(r"```\n(.*?)```", text, re.S) if "lr.Router(" in b)
    once, step = code.split("# every step\n")
    return once, step


def test_readme_training_step():
    once, step = _example()
    T, E, K, D, F = 257, 5, 2, 128, 64
    rng = np.random.default_rng(31)

    def bf(*shape, std=1.0):
        return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(DEV).bfloat16()

    W1, W2 = bf(E, D, 2 * F, std=D ** -0.5), bf(E, F, D, std=F ** -0.5)
    env = {"lr": lr, "T": T, "E": E, "K": K, "D": D, "F": F, "W1": W1, "W2": W2, "M1": W1.float(), "M2": W2.float(),
           "quotas": lambda seg_off: np.diff(seg_off).astype(np.int32)}
    masters = [env["M1"].clone(), env["M2"].clone()]
    twin = lr.AdamW([W1.clone(), W2.clone()], masters=masters, lr=3e-4, bits=8)

    def inputs():
        env.update(X=bf(T, D), G=bf(T, D), logits=torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV),
                   mask=torch.from_numpy(rng.random(T) < 0.9).to(DEV))

    log("what the README runs once")
    inputs()
    exec(once, env)
    for i in range(3):
        inputs()
        log(f"the README's step {i}")
        exec(step, env)
        g = env["g"]
        twin.step([g["dW1"].clone(), g["dW2"].clone()])
        torch.cuda.synchronize()
        assert torch.equal(env["M1"], masters[0]) and torch.equal(env["M2"], masters[1]), i
        assert torch.equal(W1, twin.w[0]) and torch.equal(W2, twin.w[1]), i
        assert env["dlogits"].shape == (T, E) and env["y"].shape == (T, D) and float(env["b"]["loss"]) > 0
        g["dW1"].fill_(7.0)  # if a later step used these again
        g["dW2"].fill_(7.0)
