"""A residual block under a vocabulary head, trained by plain gradient descent on random tokens.

    b = x @ W1                                   the block: a GEMM of this library
    y = x + alpha gate N_post(b) w_post          gemm_epi_norm_run, which also gives
    h = N_pre(y) w_pre                           the hidden states of the head
    loss = cross entropy of h against W          gemm_epi_xent_step, which also gives dh and dW
    db, dgate, dw_post, dw_pre                   gemm_epi_norm_grad
    dW1 = x^T @ db                               a GEMM on column-major A

    python examples/train_block.py [--steps 30] [--tokens 512] [--width 256] [--vocabulary 1000]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dense_gemm_elementwise_gb300 import binding as B  # noqa: E402

DAG = [("accum", 0, 0, 0), ("store", 0, 0, 0)]  # D = A @ B


class Model:
    """Plans, parameters, workspaces and gradient buffers for batches of `tokens` rows."""

    def __init__(self, tokens, width, vocabulary, alpha=0.5, seed=0):
        T, D, V = tokens, width, vocabulary
        dev, dt = torch.device("cuda", 0), torch.bfloat16
        g = torch.Generator(device=dev)
        g.manual_seed(seed)

        def randn(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device=dev) * scale).to(dt)

        def empty(*shape, dtype=dt):
            return torch.empty(*shape, dtype=dtype, device=dev)

        self.alpha = alpha
        self.p = {"W1": randn(D, D, scale=D ** -0.5), "W": randn(V, D, scale=D ** -0.5), "gate": torch.ones(1, D, dtype=dt, device=dev),
                  "w_post": torch.ones(D, dtype=dt, device=dev), "w_pre": torch.ones(D, dtype=dt, device=dev)}
        self.grad = {k: torch.empty_like(v) for k, v in self.p.items()}
        # master weights in 32 bits: bf16 alone loses small steps
        self.master = {k: v.float() for k, v in self.p.items()}
        self.embed = randn(V, D)
        types = B.make_dtypes("bf16", [], 0, ["bf16"])
        self.block = B.gemm_epi_plan_create(1, T, D, D, types, B.make_dag(DAG))
        columns = B.ge_options()
        columns.a_major = B.GE_COL_MAJOR
        self.block_grad = B.gemm_epi_plan_create(1, D, D, T, types, B.make_dag(DAG), columns)
        self.norm = B.gemm_epi_norm_plan_create(T, D, B.make_norm_desc("bf16", "bf16", alpha=alpha, rows_per_gate=T))
        self.head = B.gemm_epi_xent_plan_create(T, V, D, B.make_xent_desc("bf16", reduction="mean"))
        self.norm_ws = empty(B.gemm_epi_norm_workspace_bytes(self.norm), dtype=torch.uint8)
        self.head_ws = empty(B.gemm_epi_xent_workspace_bytes(self.head, True), dtype=torch.uint8)
        self.b, self.y, self.h, self.dh, self.dx, self.db = (empty(T, D) for _ in range(6))
        self.loss, self.lse, self.total = (empty(n, dtype=torch.float32) for n in (T, T, 1))

    def step(self, x, target):
        """The loss of one batch (a device scalar) and, in self.grad, its gradients."""
        p, g = self.p, self.grad
        B.gemm_epi_run(self.block, x, p["W1"], [], [], [self.b])
        B.gemm_epi_norm_run(self.norm, x, self.b, p["gate"], p["w_post"], p["w_pre"], self.y, self.h)
        B.gemm_epi_xent_step(self.head, self.h, p["W"], target, None, 1.0, self.loss, self.lse, self.total, self.dh, g["W"],
                             self.head_ws)
        B.gemm_epi_norm_grad(self.norm, None, self.dh, self.y, self.b, p["gate"], p["w_post"], p["w_pre"], self.dx, self.db,
                             g["gate"], g["w_post"], g["w_pre"], self.norm_ws)
        B.gemm_epi_run(self.block_grad, x, self.db, [], [], [g["W1"]])
        return self.total

    def descend(self, rate):
        for k, v in self.master.items():
            v.sub_(self.grad[k].float(), alpha=rate)
            self.p[k].copy_(v)

    def close(self):
        B.gemm_epi_plan_destroy(self.block)
        B.gemm_epi_plan_destroy(self.block_grad)
        B.gemm_epi_norm_plan_destroy(self.norm)
        B.gemm_epi_xent_plan_destroy(self.head)


def train(steps, tokens, width, vocabulary, rate=1.0, seed=0):
    """Losses of `steps` steps on one batch: token i is to predict a fixed permutation of itself; a tenth are ignored."""
    m = Model(tokens, width, vocabulary, seed=seed)
    dev = m.embed.device
    g = torch.Generator(device=dev)
    g.manual_seed(seed + 1)
    ids = torch.randint(0, vocabulary, (tokens,), generator=g, device=dev)
    target = (ids * 7 + 3) % vocabulary
    target[::10] = -100
    x = m.embed[ids].contiguous()
    losses = []
    for _ in range(steps):
        losses.append(m.step(x, target).clone())
        m.descend(rate)
    torch.cuda.synchronize()
    status = B.gemm_epi_last_error()
    m.close()
    if status != B.GE_OK:
        raise RuntimeError("device status " + B.gemm_epi_status_string(status))
    return [float(v) for v in losses]


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    a.add_argument("--steps", type=int, default=30)
    a.add_argument("--tokens", type=int, default=512)
    a.add_argument("--width", type=int, default=256)
    a.add_argument("--vocabulary", type=int, default=1000)
    a = a.parse_args()
    for i, v in enumerate(train(a.steps, a.tokens, a.width, a.vocabulary)):
        print("step %3d  loss %.4f" % (i, v))
