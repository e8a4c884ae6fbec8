"""The operators of the fp8 layer and the token read-out together, as examples/fp8_readout.py runs them.

Tolerance against the same network in fp32 without quantization, on the 2-norm of the logits: a code is off by at
most 2^-4 of its value, uniformly within its step: at most 2^-4 / sqrt 3 = 3.6% rms.  A product of two quantized
operands is off by 5.1%; h is a product of two such, 7.2%, and quantized and multiplied again 8.9%; the hidden states
added to it dilute that, the head's product brings it to at most 10.3%.  15% leaves room for what is not uniform.
"""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))
import fp8_readout  # noqa: E402
from gpu_util import DEV  # noqa: E402

pytestmark = pytest.mark.gpu

H, I, V = 400, 1040, 9001


def weights():
    g = torch.Generator(device=DEV).manual_seed(3)
    return [torch.randn(s, generator=g, device=DEV) * s[1] ** -0.5 for s in ((2 * I, H), (H, I), (V, H))]


@pytest.mark.parametrize("m", [1, 5, 70])
def test_step(m):
    gate_up, down, head = weights()
    model = fp8_readout.Readout(gate_up, down, head * 4)
    g = torch.Generator(device=DEV).manual_seed(m)
    x = torch.randn((m, H), generator=g, device=DEV)
    answers = torch.randint(0, V, (m, 6), generator=g, device=DEV)
    choice, score, r = model(x, answers, top=5)

    gu = (x.double() @ gate_up.double().t().contiguous()).cpu().numpy()
    h = gu[:, :I] / (1 + np.exp(-gu[:, :I])) * gu[:, I:]
    y = x.double().cpu().numpy() + h @ down.double().cpu().numpy().T
    plain = y @ head.double().cpu().numpy().T * 4
    z = model.logits(x).double().cpu().numpy()
    assert np.linalg.norm(z - plain) <= 0.15 * np.linalg.norm(plain)

    lse = np.log(np.exp(z).sum(1))
    a = answers.cpu().numpy()
    lp = np.take_along_axis(z, a, 1) - lse[:, None]
    assert np.abs(r.logprobs.cpu().numpy() - lp).max() <= 2.0 ** -17 + 2.0 ** -22 * np.abs(lp).max()
    p = np.exp(lp) / np.exp(lp).sum(1, keepdims=True)
    assert np.abs(score.cpu().numpy() - (p * np.arange(6)).sum(1)).max() <= 1e-4  # six terms, each within 5 * 2^-16
    best = np.take_along_axis(lp, choice.cpu().numpy()[:, None], 1)[:, 0]
    assert (best >= lp.max(1) - 2.0 ** -16).all()
    for i in (0, m - 1):
        one = model(x[i:i + 1].contiguous(), answers[i:i + 1], top=5)[2]
        for u, v in zip(one, r):
            assert torch.equal(u[0], v[i])


def test_command(monkeypatch, capsys):
    monkeypatch.setattr(sys, "argv", ["fp8_readout.py", "--rows", "3", "--hidden", "272", "--inner", "528", "--vocab",
                                      "5001", "--steps", "3"])
    assert fp8_readout.main() == 0
    assert "same bits: True; row 0 alone same bits: True" in capsys.readouterr().out
