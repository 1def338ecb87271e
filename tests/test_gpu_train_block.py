"""The GEMM, the norms and the vocabulary loss together, as the training example runs them."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

from dense_gemm_elementwise_gb300 import build as gbuild  # noqa: E402

gbuild.build()
import train_block  # noqa: E402


def unit(v):
    return v / torch.sqrt(v.pow(2).mean(1, keepdim=True) + 1e-5)


@pytest.mark.gpu
def test_gradients_of_the_whole_step():
    """Against differentiation in 64 bits.  The chain rounds b, y, h, dl, dh, db and each gradient to bf16 (2^-8
    each, independent): in the 2-norm a gradient is off by less than 6 of them."""
    T, D, V = 300, 128, 501
    m = train_block.Model(T, D, V, seed=3)
    dev = m.embed.device
    ids = torch.arange(T, device=dev) * 13 % V
    target = (ids * 7 + 3) % V
    target[::10] = -100
    x = m.embed[ids].contiguous()
    total = m.step(x, target)
    torch.cuda.synchronize()
    p = {k: v.double().requires_grad_() for k, v in m.p.items()}
    xd = x.double()
    y = xd + m.alpha * p["gate"] * unit(xd @ p["W1"]) * p["w_post"]
    logits = (unit(y) * p["w_pre"]) @ p["W"].T
    want = torch.nn.functional.cross_entropy(logits, target, ignore_index=-100)
    want.backward()
    want = want.item()
    assert abs(float(total) - want) <= 2.0 ** -8 * want
    for k, v in p.items():
        off = float((m.grad[k].double() - v.grad).norm() / v.grad.norm())
        assert off <= 6 * 2.0 ** -8, (k, off)
    m.close()


@pytest.mark.gpu
def test_the_loss_falls():
    losses = train_block.train(steps=20, tokens=384, width=128, vocabulary=300)
    assert all(b < a for a, b in zip(losses[:5], losses[1:6])) and losses[-1] < 0.5 * losses[0], losses
