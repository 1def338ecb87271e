"""The language-model operators beside the fused GEMM, as they are measured.

Four passes: the vocabulary loss of a batch of hidden states (scoring), the same loss with the gradients of
the hidden states and of the vocabulary weights (a training step's head), the norms around a block fused with its gate and
residual scale, and the gradients of those norms.  `run` computes a pass in its plain form (elementary torch
operations in 32 bits, rounded once at the end) or, with `own` set, by the library's calls.
"""
import math

import torch

own = False

DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
LARGEST_MACS = 8192 * 65536 * 4096  # tokens x vocabulary x width of the largest listed step
LARGEST_ROWS = 16384 * 4096         # elements of the largest listed norm


def listed():
    return [
        # one new token scored against a whole vocabulary: latency, and the weights read once
        dict(name="loss_one_token", op="loss", T=1, V=32000, D=1024, ab="bf16", pad=0, ignored=0.0, weights=False,
             z=0.0, scale=1.0, mean=True),
        # a handful of drafted tokens, a vocabulary and a width that fill no tile
        dict(name="loss_few_odd", op="loss", T=37, V=50001, D=2001, ab="f16", pad=15, ignored=0.1, weights=True,
             z=0.0, scale=0.5, mean=False),
        # evaluation of a long batch
        dict(name="loss_eval", op="loss", T=4096, V=65536, D=2048, ab="bf16", pad=0, ignored=0.0, weights=False,
             z=0.0, scale=1.0, mean=True),
        # the smallest training step: launches count
        dict(name="step_small", op="step", T=64, V=8192, D=512, ab="f16", pad=0, ignored=0.0, weights=False,
             z=0.0, scale=1.0, mean=True),
        # fine-tuning on answers: two fifths of the targets ignored, weighted rows, a log-normaliser penalty, odd sizes
        dict(name="step_masked_odd", op="step", T=1777, V=32001, D=1280, ab="bf16", pad=0, ignored=0.4, weights=True,
             z=1e-3, scale=1.0, mean=True),
        # an ordinary pretraining step's head
        dict(name="step_ordinary", op="step", T=4096, V=32000, D=2048, ab="bf16", pad=0, ignored=0.0, weights=False,
             z=0.0, scale=1.0, mean=True),
        # a large model's: exponentials for every pair of token and word no longer fit the default workspace
        dict(name="step_large", op="step", T=8192, V=65536, D=4096, ab="bf16", pad=0, ignored=0.02, weights=False,
             z=1e-4, scale=1.0, mean=True),
        # one token between two layers of a decoder
        dict(name="norm_one_token", op="norm", T=1, D=4096, x="bf16", w="bf16", pre="rms", post="rms", gate=1, pad=0,
             alpha=1.0),
        # a prompt, gated per channel
        dict(name="norm_prompt", op="norm", T=8192, D=4096, x="bf16", w="bf16", pre="rms", post="rms", gate=8192, pad=0,
             alpha=0.7),
        # centred norms, an odd width whose rows are not whole 16-byte units, no norm on the block's output
        dict(name="norm_odd", op="norm", T=3001, D=1111, x="f16", w="f32", pre="layer", post="none", gate=0, pad=0,
             alpha=1.0),
        # gradients of a short batch in 32 bits with a gate for every token
        dict(name="norm_grad_tokens", op="norm_grad", T=333, D=1024, x="f32", w="f32", pre="layer", post="rms", gate=1,
             pad=0, alpha=0.5),
        # gradients of a training batch of eight sequences, each with its own gate
        dict(name="norm_grad_batch", op="norm_grad", T=16384, D=4096, x="bf16", w="bf16", pre="rms", post="rms",
             gate=2048, pad=0, alpha=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["loss", "step", "norm", "norm_grad"])
    if op in ("loss", "step"):
        while True:
            T, V, D = _log(rng, 1, 8192), _log(rng, 500, 131072), _log(rng, 64, 4096)
            if rng.random() < 0.5:
                D = max(8, D // 8 * 8)
            if T * V * D <= LARGEST_MACS:
                break
        return dict(op=op, T=T, V=V, D=D, ab=rng.choice(["f16", "bf16"]), pad=-D % 8 + 8 * rng.choice([0, 0, 3]),
                    ignored=rng.choice([0.0, 0.0, 0.1, 0.5, 0.9]), weights=rng.random() < 0.3,
                    z=rng.choice([0.0, 0.0, 1e-4, 1e-3]), scale=rng.choice([1.0, 1.0, 0.5]),
                    mean=rng.random() < 0.7)
    while True:
        T, D = _log(rng, 1, 16384), _log(rng, 64, 16384)
        if rng.random() < 0.5:
            D = max(8, D // 8 * 8)
        if T * D <= LARGEST_ROWS:
            break
    return dict(op=op, T=T, D=D, x=rng.choice(["f16", "bf16", "f32"]), w=rng.choice(["bf16", "f16", "f32"]),
                pre=rng.choice(["rms", "layer"]), post=rng.choice(["none", "rms", "layer"]),
                gate=rng.choice([0, 1, T, max(1, T // 7), _log(rng, 1, T)]), pad=rng.choice([0, 0, 1, 8]),
                alpha=rng.choice([1.0, 0.5, 0.125]))


# ---------------------------------------------------------------- inputs --

EPS = 1e-5


def _wide(T, D, pad, dtype, dev):
    """A (T, D) view with `pad` elements between its rows, filled with what must not matter."""
    return torch.full((T, D + pad), 7.0, dtype=dtype, device=dev)[:, :D]


def _put(x, pad, dtype):
    v = _wide(x.shape[0], x.shape[1], pad, dtype, x.device)
    v.copy_(x)
    return v


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1009 + 17)
    dev = torch.device("cuda", 0)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = dict(case=case)
    if case["op"] in ("loss", "step"):
        T, V, D, dt = case["T"], case["V"], case["D"], DTYPE[case["ab"]]
        W = _put(randn(V, D).mul_(2.5 / math.sqrt(D)), case["pad"], dt)
        target = torch.randint(0, V, (T,), generator=g, device=dev)
        # normalised hidden states, half of them pointing towards their target as a trained model's do
        H = randn(T, D)
        near = torch.rand(T, 1, generator=g, device=dev) < 0.5
        H += torch.where(near, 1.0, 0.0) * W[target].float()
        H = _put(H, case["pad"], dt)
        if case["ignored"]:
            drop = torch.rand(T, generator=g, device=dev) < case["ignored"]
            target = torch.where(drop, torch.full_like(target, -100), target)
        s.update(H=H, W=W, target=target)
        s["weight"] = torch.rand(T, generator=g, device=dev) + 0.5 if case["weights"] else None
        # 16-bit floats with 5 exponent bits train with a loss scale
        s["grad_scale"] = 1024.0 if case["ab"] == "f16" else 1.0
    else:
        T, D, xt, wt, pad = case["T"], case["D"], DTYPE[case["x"]], DTYPE[case["w"]], case["pad"]
        groups = -(-T // case["gate"]) if case["gate"] else 0
        s["b"] = _put(randn(T, D) * (0.5 + 2 * torch.rand(T, 1, generator=g, device=dev)), pad, xt)
        s["gate"] = (0.5 + 0.3 * randn(groups, D)).to(wt) if groups else None
        s["w_post"] = (1 + 0.2 * randn(D)).to(wt) if case["post"] != "none" else None
        s["w_pre"] = (1 + 0.2 * randn(D)).to(wt)
        stream = _put(3 * randn(T, D) + 0.3, pad, xt)
        if case["op"] == "norm":
            s["x"] = stream
        else:
            s["y"] = stream
            s["dy"] = _put(randn(T, D), pad, xt)
            s["dh"] = _put(randn(T, D), pad, xt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _plan(s)
    return s


def _plan(s):
    """The plan, workspace and output buffers that a program using the library keeps."""
    from dense_gemm_elementwise_gb300 import binding as B
    c = s["case"]
    dev = torch.device("cuda", 0)

    def f32(*shape):
        return torch.empty(*shape, dtype=torch.float32, device=dev)

    if c["op"] in ("loss", "step"):
        T, V, D, pad, dt = c["T"], c["V"], c["D"], c["pad"], DTYPE[c["ab"]]
        desc = B.make_xent_desc(c["ab"], "i64", ldh=D + pad, ldw=D + pad, lddh=D + pad, lddw=D + pad,
                                logit_scale=c["scale"], z_loss=c["z"], reduction="mean" if c["mean"] else "sum")
        plan = B.gemm_epi_xent_plan_create(T, V, D, desc)
        step = c["op"] == "step"
        ws = torch.empty(B.gemm_epi_xent_workspace_bytes(plan, step), dtype=torch.uint8, device=dev)
        loss, lse, total = f32(T), f32(T), f32(1)
        s.update(plan=plan, ws=ws)
        if step:
            dH, dW = _wide(T, D, pad, dt, dev), _wide(V, D, pad, dt, dev)
            s["call"] = B.prepare_xent_step(plan, s["H"], s["W"], s["target"], s["weight"], s["grad_scale"], loss, lse,
                                            total, dH, dW, ws)
            s["outs"] = dict(loss=loss, lse=lse, total=total, dH=dH, dW=dW)
        else:
            s["call"] = B.prepare_xent_loss(plan, s["H"], s["W"], s["target"], s["weight"], loss, lse, total, ws)
            s["outs"] = dict(loss=loss, lse=lse, total=total)
        return
    T, D, pad, xt, wt = c["T"], c["D"], c["pad"], DTYPE[c["x"]], DTYPE[c["w"]]
    ld = D + pad
    desc = B.make_norm_desc(c["x"], c["w"], pre=c["pre"], post=c["post"], eps_pre=EPS, eps_post=EPS, alpha=c["alpha"],
                            rows_per_gate=c["gate"], ldx=ld, ldb=ld, ldy=ld, ldh=ld)
    plan = B.gemm_epi_norm_plan_create(T, D, desc)
    s["plan"] = plan
    if c["op"] == "norm":
        y, h = _wide(T, D, pad, xt, dev), _wide(T, D, pad, xt, dev)
        s["call"] = B.prepare_norm_run(plan, s["x"], s["b"], s["gate"], s["w_post"], s["w_pre"], y, h)
        s["outs"] = dict(y=y, h=h)
        return
    outs = dict(dx=_wide(T, D, pad, xt, dev), db=_wide(T, D, pad, xt, dev), dw_pre=torch.empty(D, dtype=wt, device=dev))
    if s["gate"] is not None:
        outs["dgate"] = torch.empty_like(s["gate"])
    if s["w_post"] is not None:
        outs["dw_post"] = torch.empty(D, dtype=wt, device=dev)
    s["ws"] = torch.empty(B.gemm_epi_norm_workspace_bytes(plan), dtype=torch.uint8, device=dev)
    s["call"] = B.prepare_norm_grad(plan, s["dy"], s["dh"], s["y"], s["b"], s["gate"], s["w_post"], s["w_pre"],
                                    outs["dx"], outs["db"], outs.get("dgate"), outs.get("dw_post"), outs["dw_pre"],
                                    s["ws"])
    s["outs"] = outs


# ------------------------------------------------------------------ run --

def run(s):
    if own:
        status = s["call"]()
        if status:
            raise RuntimeError("status %d" % status)
        return s["outs"]
    return PLAIN[s["case"]["op"]](s)


def _plain_xent(s, grads):
    c = s["case"]
    H, W, t = s["H"].float(), s["W"].float(), s["target"]
    valid = (t >= 0) & (t < c["V"])
    tt = torch.where(valid, t, torch.zeros_like(t))
    w = s["weight"] if s["weight"] is not None else torch.ones(c["T"], device=H.device)
    w = torch.where(valid, w, torch.zeros_like(w))
    p = (H @ W.T).mul_(c["scale"])
    top = p.max(1, keepdim=True).values
    at = p.gather(1, tt[:, None])
    p = p.sub_(top).exp_()
    total = p.sum(1, keepdim=True)
    lse = top + total.log()
    row = (lse - at + c["z"] * lse * lse)[:, 0]
    none = torch.zeros_like(row)
    row = torch.where(valid, row * w, none)
    norm = w.sum() if c["mean"] else torch.ones((), device=H.device)
    whole = torch.where(norm != 0, row.sum() / norm, torch.zeros_like(norm)).reshape(1)
    out = dict(loss=row, lse=torch.where(valid, lse[:, 0], none), total=whole)
    if grads:
        g = torch.where(norm != 0, w * s["grad_scale"] / norm, none)[:, None]
        p = p.mul_((1 + 2 * c["z"] * lse) / total * g)
        p.scatter_add_(1, tt[:, None], -g)
        p = p.mul_(c["scale"])
        out["dH"] = (p @ W).to(DTYPE[c["ab"]])
        out["dW"] = (p.T @ H).to(DTYPE[c["ab"]])
    return out


def _unit(v, kind):
    """The rows of v over their root mean square or, centred, over their standard deviation; and that divisor's inverse."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = ((v * v).mean(1, keepdim=True) + EPS).rsqrt()
    return v * r, r


def _unit_grad(d, u, r, kind):
    """The gradient through _unit: `d` of its outputs u, whose inverse divisor is r."""
    d = d - u * (d * u).mean(1, keepdim=True) if kind != "layer" else \
        d - d.mean(1, keepdim=True) - u * (d * u).mean(1, keepdim=True)
    return d * r


def _rows_of_gate(s):
    c = s["case"]
    at = torch.arange(c["T"], device=s["b"].device) // c["gate"]
    return s["gate"].float()[at], at


def _plain_norm(s):
    c = s["case"]
    x, b = s["x"].float(), s["b"].float()
    if c["post"] != "none":
        b = _unit(b, c["post"])[0] * s["w_post"].float()
    if s["gate"] is not None:
        b = b * _rows_of_gate(s)[0]
    y = x + c["alpha"] * b
    h = _unit(y, c["pre"])[0] * s["w_pre"].float()
    xt = DTYPE[c["x"]]
    return dict(y=y.to(xt), h=h.to(xt))


def _plain_norm_grad(s):
    c = s["case"]
    xt, wt = DTYPE[c["x"]], DTYPE[c["w"]]
    dy, dh, y, b = s["dy"].float(), s["dh"].float(), s["y"].float(), s["b"].float()
    u, r = _unit(y, c["pre"])
    dt = dy + _unit_grad(dh * s["w_pre"].float(), u, r, c["pre"])
    out = dict(dx=dt.to(xt), dw_pre=(dh * u).sum(0).to(wt))
    n, rp = _unit(b, c["post"]) if c["post"] != "none" else (b, None)
    d = c["alpha"] * dt
    wp = s["w_post"].float() if s["w_post"] is not None else 1.0
    if s["gate"] is not None:
        gate, at = _rows_of_gate(s)
        dgate = torch.zeros(s["gate"].shape, device=b.device)
        dgate.index_add_(0, at, d * n * wp)
        out["dgate"] = dgate.to(wt)
        d = d * gate
    if s["w_post"] is not None:
        out["dw_post"] = (d * n).sum(0).to(wt)
        d = _unit_grad(d * wp, n, rp, c["post"])
    out["db"] = d.to(xt)
    return out


PLAIN = {"loss": lambda s: _plain_xent(s, False), "step": lambda s: _plain_xent(s, True), "norm": _plain_norm,
         "norm_grad": _plain_norm_grad}


# ----------------------------------------------------------------- exact --

def exact(case, seed):
    if case["op"] in ("loss", "step"):
        macs = case["T"] * case["V"] * case["D"] * (3 if case["op"] == "step" else 1)
        if macs > 8e12:  # 64-bit products of this size take over 20 seconds
            return None
        return _exact_xent(case, _inputs(case, seed))
    return _exact_norm(case, _inputs(case, seed))


def _exact_xent(c, s):
    """Rows of tokens one block at a time: L_i = w_i (lse_i - l_i,t + z lse_i^2), its derivative by every logit, and the
    two products of that derivative."""
    T, V, D = c["T"], c["V"], c["D"]
    W = s["W"].double()
    dev = W.device
    loss = torch.zeros(T, dtype=torch.float64, device=dev)
    lse = torch.zeros_like(loss)
    w = torch.ones_like(loss) if s["weight"] is None else s["weight"].double()
    keep = ((s["target"] >= 0) & (s["target"] < V)).nonzero()[:, 0]
    norm = float(w[keep].sum()) if c["mean"] else 1.0
    grads = c["op"] == "step"
    dH = torch.zeros(T, D, dtype=torch.float64, device=dev)
    dW = torch.zeros(V, D, dtype=torch.float64, device=dev) if grads else None
    for i in range(0, keep.numel(), 1024):
        at = keep[i:i + 1024]
        h, t = s["H"][at].double(), s["target"][at]
        logit = c["scale"] * (h @ W.T)
        n = torch.logsumexp(logit, 1)
        lse[at] = n
        loss[at] = w[at] * (n - logit[torch.arange(at.numel(), device=dev), t] + c["z"] * n ** 2)
        if grads and norm:
            d = torch.softmax(logit, 1) * (1 + 2 * c["z"] * n)[:, None]
            d[torch.arange(at.numel(), device=dev), t] -= 1
            d *= (w[at] * (s["grad_scale"] * c["scale"] / norm))[:, None]
            dH[at] = d @ W
            dW += d.T @ h
    out = dict(loss=loss, lse=lse, total=(loss.sum() / norm if norm else loss.sum() * 0).reshape(1))
    if grads:
        out.update(dH=dH, dW=dW)
    return out


def _exact_norm(c, s):
    """By torch's differentiation in 64 bits of the definition, as one function of the stream and the block's output."""
    T, D = c["T"], c["D"]
    par = {k: s[k].double().requires_grad_() for k in ("b", "gate", "w_post", "w_pre") if s.get(k) is not None}
    rows = None if s["gate"] is None else torch.arange(T, device=s["b"].device).div(c["gate"], rounding_mode="floor")

    def unit(v, kind):
        if kind == "none":
            return v
        if kind == "layer":
            return (v - v.mean(1, keepdim=True)) / torch.sqrt(v.var(1, unbiased=False, keepdim=True) + EPS)
        return v / torch.sqrt(v.pow(2).mean(1, keepdim=True) + EPS)

    def branch():
        v = unit(par["b"], c["post"])
        if "w_post" in par:
            v = v * par["w_post"]
        if rows is not None:
            v = v * par["gate"][rows]
        return c["alpha"] * v

    if c["op"] == "norm":
        with torch.no_grad():
            y = s["x"].double() + branch()
            return dict(y=y, h=unit(y, c["pre"]) * par["w_pre"])
    y = s["y"].double().requires_grad_()
    wrt = [y, par["w_pre"]]
    dpre = torch.autograd.grad((unit(y, c["pre"]) * par["w_pre"] * s["dh"].double()).sum(), wrt)
    dx = dpre[0] + s["dy"].double()
    names = [k for k in ("b", "gate", "w_post") if k in par]
    got = dict(zip(names, torch.autograd.grad((branch() * dx).sum(), [par[k] for k in names])))
    out = dict(dx=dx, dw_pre=dpre[1], db=got["b"])
    if "gate" in got:
        out["dgate"] = got["gate"]
    if "w_post" in got:
        out["dw_post"] = got["w_post"]
    return out


# ------------------------------------------------------------------ work --

def work(c):
    T, D = c["T"], c["D"]
    if c["op"] in ("loss", "step"):
        V = c["V"]
        rows = round(T * (1 - c["ignored"]))  # an ignored target's row needs no product
        io = 2 * (rows * D + V * D) + T * (8 + 8 + (4 if c["weights"] else 0))
        if c["op"] == "loss":
            return dict(bytes=io, flops=2 * rows * V * D)
        return dict(bytes=io + 2 * (T * D + V * D), flops=6 * rows * V * D)
    ex, ew = (2 if c["x"] != "f32" else 4), (2 if c["w"] != "f32" else 4)
    groups = -(-T // c["gate"]) if c["gate"] else 0
    vec = (groups + 1 + (c["post"] != "none")) * D * ew
    if c["op"] == "norm":
        return dict(bytes=4 * T * D * ex + vec, flops=12 * T * D)
    return dict(bytes=6 * T * D * ex + 2 * vec, flops=30 * T * D)
