"""Products of 8-bit floats with a scale for each block of 128, and a mixture-of-experts layer for a few tokens, as
they are measured.

Three passes: values and scales made from a matrix (`quant`), the scaled product (`fp8`), and a whole layer of experts
with its router (`moe`).  `run` computes a pass in its plain form (elementary torch operations in 32 bits, the router's
logits in 64, rounded once at the end) or, with `own` set, by the library's calls.
"""
import math

import torch

own = False

DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
         "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
SMALLEST_SCALE = 2.0 ** -126
BLOCK = 128
LARGEST_QUANT = 16384 * 4096           # elements of the largest listed matrix
LARGEST_MACS = 8192 ** 3               # of the largest listed product
LARGEST_EXPERTS = 128 * 3 * 4096 * 2048  # bytes of the largest listed layer's experts


def listed():
    return [
        # one new token's hidden state: latency
        dict(name="quant_token", op="quant", T=1, D=4096, x="bf16", q="e4m3", block="row", rows=True, cols=False,
             pad=0),
        # a training batch's activations, for the forward product and, transposed, for the weights' gradient
        dict(name="quant_batch", op="quant", T=16384, D=4096, x="bf16", q="e4m3", block="row", rows=True, cols=True,
             pad=0),
        # master weights after an optimizer's step, in squares, both orders; no size a multiple of a block
        dict(name="quant_weights_odd", op="quant", T=5001, D=2730, x="f32", q="e4m3", block="square", rows=True,
             cols=True, pad=2),
        # one new token through a linear layer: the weights read once
        dict(name="fp8_one_token", op="fp8", M=1, N=8192, K=4096, a="e4m3", b="e4m3", block="square", out="bf16",
             add=False, pad=0),
        # drafted tokens, sizes that fill no tile
        dict(name="fp8_few_odd", op="fp8", M=37, N=5001, K=2000, a="e4m3", b="e4m3", block="square", out="f16",
             add=False, pad=16),
        # a prompt through a linear layer
        dict(name="fp8_prompt", op="fp8", M=4096, N=4096, K=4096, a="e4m3", b="e4m3", block="square", out="bf16",
             add=False, pad=0),
        # gradients of the weights summed over micro-batches in 32 bits: both operands scaled along the tokens
        dict(name="fp8_weight_gradient", op="fp8", M=4096, N=2048, K=6001, a="e5m2", b="e4m3", block="row", out="f32",
             add=True, pad=15),
        # a large product
        dict(name="fp8_large", op="fp8", M=8192, N=8192, K=8192, a="e4m3", b="e4m3", block="square", out="bf16",
             add=False, pad=0),
        # one token of a decoder: latency, and a few experts' weights
        dict(name="moe_one_token", op="moe", T=1, D=2048, F=1024, E=64, k=8, x="bf16", w="bf16", score="softmax",
             norm=True, bias=False, scale=1.0),
        # a small batch of sequences, one token each
        dict(name="moe_batch", op="moe", T=8, D=4096, F=1536, E=32, k=4, x="bf16", w="bf16", score="softmax", norm=True,
             bias=False, scale=1.0),
        # drafted tokens of several sequences, odd sizes, a choice balanced by a bias
        dict(name="moe_odd", op="moe", T=29, D=1000, F=520, E=13, k=3, x="f16", w="f16", score="sigmoid", norm=True,
             bias=True, scale=2.5),
        # a large layer whose weights are held in 8 bits: nearly every expert is read for a handful of tokens
        dict(name="moe_large_8bit", op="moe", T=64, D=4096, F=2048, E=128, k=8, x="bf16", w="e4m3", score="sigmoid",
             norm=True, bias=True, scale=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "fp8", "moe"])
    if op == "quant":
        while True:
            T, D = _log(rng, 1, 16384), _log(rng, 64, 16384)
            if rng.random() < 0.5:
                D = max(16, D // 16 * 16)
            if T * D <= LARGEST_QUANT:
                break
        rows, cols = rng.choice([(True, False), (False, True), (True, True)])
        return dict(op=op, T=T, D=D, x=rng.choice(["f16", "bf16", "f32"]), q=rng.choice(["e4m3", "e4m3", "e5m2"]),
                    block=rng.choice(["row", "row", "square"]), rows=rows, cols=cols, pad=rng.choice([0, 0, 8]))
    if op == "fp8":
        while True:
            M, N, K = _log(rng, 1, 8192), _log(rng, 64, 16384), _log(rng, 64, 16384)
            if rng.random() < 0.6:
                N, K = max(64, N // 64 * 64), max(64, K // 64 * 64)
            if M * N * K <= LARGEST_MACS:
                break
        out = rng.choice(["bf16", "bf16", "f16", "f32"])
        a, b = rng.choice(["e4m3", "e4m3", "e5m2"]), rng.choice(["e4m3", "e4m3", "e5m2"])
        return dict(op=op, M=M, N=N, K=K, a=a, b=b, block=rng.choice(["square", "square", "row"]), out=out,
                    add=rng.random() < 0.3, pad=-K % 16 + rng.choice([0, 0, 16]))
    while True:
        T, D, F, E = _log(rng, 1, 64), _log(rng, 256, 8192), _log(rng, 128, 4096), _log(rng, 4, 256)
        D, F = D // 8 * 8, F // 8 * 8
        x = rng.choice(["f16", "bf16"])
        w = rng.choice([x, x, "e4m3"])
        if w == "e4m3":
            D, F = D // 16 * 16, F // 16 * 16
        if E * 3 * D * F * (1 if w == "e4m3" else 2) <= LARGEST_EXPERTS:
            break
    return dict(op=op, T=T, D=D, F=F, E=E, k=rng.randint(1, min(8, E)), x=x, w=w,
                score=rng.choice(["softmax", "sigmoid"]), norm=rng.random() < 0.7, bias=rng.random() < 0.4,
                scale=rng.choice([1.0, 1.0, 2.5]))


# ---------------------------------------------------------------- inputs --

def _blocks(n):
    return -(-n // BLOCK)


def _up(n, m):
    return -(-n // m) * m


def _wide(rows, cols, pitch, dtype, dev):
    """A (rows, cols) view of rows `pitch` elements apart."""
    return torch.zeros(rows, pitch, dtype=torch.uint8 if dtype in (DTYPE["e4m3"], DTYPE["e5m2"]) else dtype,
                       device=dev).view(dtype)[:, :cols]


def _values(x, kind):
    """8-bit floats of numbers that are within their range."""
    return x.clamp_(-LARGEST[kind], LARGEST[kind]).to(DTYPE[kind])


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1009 + 29)
    dev = torch.device("cuda", 0)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    def eight(rows, cols, pitch, kind):
        # what the quantiser leaves: the largest of a block near the type's largest
        v = _wide(rows, cols, pitch, DTYPE[kind], dev)
        v.view(torch.uint8).copy_(_values(randn(rows, cols).mul_(LARGEST[kind] / 3.5), kind).view(torch.uint8))
        return v

    def scales(*shape):
        return (randn(*shape) * 0.5 - 4).exp()

    s = dict(case=case)
    if case["op"] == "quant":
        # activations and weights as they come: rows and columns of different magnitudes, a few outliers
        T, D, pad = case["T"], case["D"], case["pad"]
        x = randn(T, D).mul_((randn(T, 1)).exp()).mul_((0.5 * randn(1, D)).exp())
        v = _wide(T, D, D + pad, DTYPE[case["x"]], dev)
        s["x"] = v.copy_(x.clamp_(-6e4, 6e4))
    elif case["op"] == "fp8":
        M, N, K, pad = case["M"], case["N"], case["K"], case["pad"]
        s["A"], s["B"] = eight(M, K, K + pad, case["a"]), eight(N, K, K + pad, case["b"])
        s["sa"] = scales(_blocks(K), _up(M, 4))[:, :M]
        s["sb"] = scales(_blocks(K), _up(N, 4))[:, :N] if case["block"] == "row" else scales(_blocks(K), _blocks(N))
        if case["add"]:
            s["C"] = (randn(M, N) * 50 * math.sqrt(K)).to(DTYPE[case["out"]])
    else:
        T, D, F, E, xt = case["T"], case["D"], case["F"], case["E"], DTYPE[case["x"]]
        s["x"] = randn(T, D).to(xt)
        s["router"] = randn(E, D).mul_(D ** -0.5).to(xt)
        s["bias"] = 0.1 * randn(E) if case["bias"] else None
        for name, rows, cols in (("up", 2 * F, D), ("down", D, F)):
            w = torch.empty(E, rows, cols, dtype=DTYPE[case["w"]], device=dev)
            some = max(1, (1 << 28) // (rows * cols))  # at a time
            for e in range(0, E, some):
                v = randn(min(some, E - e), rows, cols)
                if case["w"] == "e4m3":
                    w[e:e + some].view(torch.uint8).copy_(_values(v.mul_(128.0), "e4m3").view(torch.uint8))
                else:
                    w[e:e + some] = v.mul_(cols ** -0.5)
            s[name] = w
            s["s_" + name] = None
            if case["w"] == "e4m3":
                s["s_" + name] = (0.5 + rand(E, _blocks(cols), _blocks(rows))) * (cols ** -0.5 / 128)
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

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=dev)

    if c["op"] == "quant":
        T, D = c["T"], c["D"]
        row = c["block"] == "row"
        desc = B.make_quant_desc(c["x"], c["q"], block=c["block"], ldx=D + c["pad"], ldq=_up(D, 16), ldqt=_up(T, 16),
                                 lds=_up(T, 4) if row else 0, ldst=_up(D, 4) if row else 0)
        s["plan"] = plan = B.gemm_epi_quant_plan_create(T, D, desc)
        outs = {}
        if c["rows"]:
            outs["q"] = _wide(T, D, _up(D, 16), DTYPE[c["q"]], dev)
            outs["scale"] = empty(_blocks(D), _up(T, 4))[:, :T] if row else empty(_blocks(D), _blocks(T))
        if c["cols"]:
            outs["qt"] = _wide(D, T, _up(T, 16), DTYPE[c["q"]], dev)
            outs["scale_t"] = empty(_blocks(T), _up(D, 4))[:, :D] if row else empty(_blocks(T), _blocks(D))
        s["call"] = B.prepare_quant_run(plan, s["x"], outs.get("q"), outs.get("scale"), outs.get("qt"),
                                        outs.get("scale_t"))
    elif c["op"] == "fp8":
        M, N, K = c["M"], c["N"], c["K"]
        desc = B.make_fp8_desc(c["a"], c["b"], c["out"], b_block=c["block"], lda=K + c["pad"], ldb=K + c["pad"],
                               lds_a=_up(M, 4), lds_b=_up(N, 4) if c["block"] == "row" else 0)
        s["plan"] = plan = B.gemm_epi_fp8_plan_create(M, N, K, desc)
        s["ws"] = empty(max(1, B.gemm_epi_fp8_workspace_bytes(plan)), dtype=torch.uint8)
        outs = dict(D=empty(M, N, dtype=DTYPE[c["out"]]))
        s["call"] = B.prepare_fp8_run(plan, s["A"], s["sa"], s["B"], s["sb"], s.get("C"), outs["D"], s["ws"])
    else:
        T, D, k = c["T"], c["D"], c["k"]
        desc = B.make_moe_desc(c["x"], c["w"], c["x"], score=c["score"], renormalise=c["norm"], route_scale=c["scale"])
        s["plan"] = plan = B.gemm_epi_moe_plan_create(T, D, c["F"], c["E"], k, desc)
        s["ws"] = empty(B.gemm_epi_moe_workspace_bytes(plan), dtype=torch.uint8)
        outs = dict(y=empty(T, D, dtype=DTYPE[c["x"]]), index=empty(T, k, dtype=torch.int32), weight=empty(T, k))
        s["call"] = B.prepare_moe_run(plan, s["x"], s["router"], s["bias"], s["up"], s["s_up"], s["down"], s["s_down"],
                                      outs["y"], outs["index"], outs["weight"], s["ws"])
    s["outs"] = outs


# ------------------------------------------------------------------- run --

def run(s):
    if own:
        status = s["call"]()
        if status:
            raise RuntimeError("status %d" % status)
        return s["outs"]
    return PLAIN[s["case"]["op"]](s)


def _padded(x):
    """x with zeros up to whole blocks in both directions."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK, 0, -x.shape[0] % BLOCK))


def _eight_bits(x, inv, kind):
    return (x * inv).clamp(-LARGEST[kind], LARGEST[kind]).to(DTYPE[kind])


def _scale_of(amax, kind):
    return (amax / LARGEST[kind]).clamp_min(SMALLEST_SCALE)


def _plain_quant(s):
    c = s["case"]
    T, D, kind = c["T"], c["D"], c["q"]
    x = s["x"].float()
    p = _padded(x)
    t, d = p.shape[0] // BLOCK, p.shape[1] // BLOCK
    four = p.abs().reshape(t, BLOCK, d, BLOCK)
    out = {}
    if c["block"] == "square":
        scale = _scale_of(four.amax((1, 3)), kind)
        q = _eight_bits(x, (1 / scale).repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)[:T, :D], kind)
        if c["rows"]:
            out.update(q=q, scale=scale.t().contiguous())
        if c["cols"]:
            out.update(qt=q.t().contiguous(), scale_t=scale)
        return out
    if c["rows"]:
        scale = _scale_of(four.amax(3).reshape(t * BLOCK, d)[:T], kind)
        out.update(q=_eight_bits(x, (1 / scale).repeat_interleave(BLOCK, 1)[:, :D], kind), scale=scale.t().contiguous())
    if c["cols"]:
        scale = _scale_of(four.amax(1).reshape(t, d * BLOCK)[:, :D], kind)
        q = _eight_bits(x, (1 / scale).repeat_interleave(BLOCK, 0)[:T], kind)
        out.update(qt=q.t().contiguous(), scale_t=scale)
    return out


def _plain_fp8(s):
    c = s["case"]
    K, N = c["K"], c["N"]
    A = s["A"].float() * s["sa"].t().repeat_interleave(BLOCK, 1)[:, :K]
    sb = s["sb"] if c["block"] == "row" else s["sb"].repeat_interleave(BLOCK, 1)[:, :N]
    B = s["B"].float() * sb.t().repeat_interleave(BLOCK, 1)[:, :K]
    y = A @ B.t()
    if c["add"]:
        y = y + s["C"].float()
    return dict(D=y.to(DTYPE[c["out"]]))


def _weights(w, scale):
    """Experts' weights in 32 bits."""
    w = w.float()
    if scale is not None:
        rows, cols = w.shape[1:]
        w = w * scale.transpose(1, 2).repeat_interleave(BLOCK, 1)[:, :rows].repeat_interleave(BLOCK, 2)[:, :, :cols]
    return w


def _plain_moe(s):
    c = s["case"]
    T, F, E, k = c["T"], c["F"], c["E"], c["k"]
    logits = s["x"].double() @ s["router"].double().t()
    p = torch.softmax(logits, 1) if c["score"] == "softmax" else torch.sigmoid(logits)
    # ties go to the lowest index: a stable sort
    by = p + s["bias"].double() if c["bias"] else logits
    index = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :k]
    weight = p.gather(1, index)
    if c["norm"]:
        weight = weight / weight.sum(1, keepdim=True)
    weight = (weight * c["scale"]).float()
    x = s["x"].float()

    def some(name, at):
        scale = s["s_" + name]
        return _weights(s[name][at], None if scale is None else scale[at])

    if T * k <= E:  # the chosen experts' weights alone
        at = index.reshape(-1)
        gu = (some("up", at) @ x.repeat_interleave(k, 0)[:, :, None])[:, :, 0]
        h = torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]
        y = (some("down", at) @ h[:, :, None])[:, :, 0].reshape(T, k, -1)
        y = (y * weight[:, :, None]).sum(1)
    else:  # every expert for every token, those that were not chosen times 0
        every = torch.zeros(T, E, device=x.device).scatter_(1, index, weight)
        gu = x @ _weights(s["up"], s["s_up"]).transpose(1, 2)
        h = torch.nn.functional.silu(gu[:, :, :F]) * gu[:, :, F:]
        y = ((h @ _weights(s["down"], s["s_down"]).transpose(1, 2)) * every.t()[:, :, None]).sum(0)
    return dict(y=y.to(DTYPE[c["x"]]), index=index.int(), weight=weight)


PLAIN = {"quant": _plain_quant, "fp8": _plain_fp8, "moe": _plain_moe}


# ----------------------------------------------------------------- exact --

def exact(case, seed):
    return {"quant": _exact_quant, "fp8": _exact_fp8, "moe": _exact_moe}[case["op"]](case, _inputs(case, seed))


def _exact_quant(c, s):
    """Scales from the definition, and the numbers that the 8-bit values stand for: x over its block's scale."""
    x = s["x"].double()
    T, D = x.shape

    def over(x):  # blocks of 128 along the last dimension
        top = torch.stack([b.abs().amax(1) for b in x.split(BLOCK, 1)])
        scale = (top / LARGEST[c["q"]]).clamp_min(SMALLEST_SCALE)
        return scale, torch.cat([b / v[:, None] for b, v in zip(x.split(BLOCK, 1), scale)], 1)

    def squares(x):
        top = torch.stack([torch.stack([b.abs().max() for b in r.split(BLOCK, 0)]) for r in x.split(BLOCK, 1)])
        scale = (top / LARGEST[c["q"]]).clamp_min(SMALLEST_SCALE)
        return scale, torch.cat([torch.cat([b / v for b, v in zip(r.split(BLOCK, 0), w)], 0)
                                 for r, w in zip(x.split(BLOCK, 1), scale)], 1)

    f = over if c["block"] == "row" else squares
    out = {}
    if c["rows"]:
        out["scale"], out["q"] = f(x)
    if c["cols"]:
        out["scale_t"], out["qt"] = f(x.t())
    return out


def _exact_fp8(c, s):
    """One block of the contraction after the other."""
    y = s["C"].double() if c["add"] else torch.zeros(c["M"], c["N"], dtype=torch.float64, device=s["A"].device)
    for kb in range(_blocks(c["K"])):
        at = slice(kb * BLOCK, min(c["K"], (kb + 1) * BLOCK))
        sb = s["sb"][kb].double()
        if c["block"] == "square":
            sb = sb[torch.arange(c["N"], device=sb.device) // BLOCK]
        y = torch.addmm(y, s["A"][:, at].double() * s["sa"][kb].double()[:, None],
                        (s["B"][:, at].double() * sb[:, None]).t())
    return dict(D=y)


def _exact_moe(c, s):
    """Expert after expert, with the tokens that chose it."""
    T, F, E, k = c["T"], c["F"], c["E"], c["k"]
    x = s["x"].double()
    logits = torch.einsum("td,ed->te", x, s["router"].double())
    if c["score"] == "softmax":
        p = (logits - logits.logsumexp(1, keepdim=True)).exp()
    else:
        p = 1 / (1 + (-logits).exp())
    by = logits if s["bias"] is None else p + s["bias"].double()
    index = by.argsort(dim=1, descending=True, stable=True)[:, :k]
    weight = torch.stack([p[t, index[t]] for t in range(T)])
    if c["norm"]:
        weight = weight / weight.sum(1)[:, None]
    weight = weight * c["scale"]
    y = torch.zeros(T, c["D"], dtype=torch.float64, device=x.device)

    def of(name, e):
        w = s[name][e].double()
        if s["s_" + name] is None:
            return w
        r, q = (torch.arange(n, device=w.device) // BLOCK for n in w.shape)
        return w * s["s_" + name][e].double()[q][:, r].t()

    for e in range(E):
        t, j = (index == e).nonzero(as_tuple=True)
        if t.numel():
            g, u = (x[t] @ of("up", e).t()).split(F, 1)
            y.index_add_(0, t, ((g / (1 + (-g).exp()) * u) @ of("down", e).t()) * weight[t, j][:, None])
    return dict(y=y, index=index.int(), weight=weight)


# ------------------------------------------------------------------ work --

SIZE = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1, "e5m2": 1}


def work(c):
    if c["op"] == "quant":
        T, D = c["T"], c["D"]
        per = BLOCK if c["block"] == "row" else BLOCK * BLOCK
        outs = c["rows"] + c["cols"]
        return dict(bytes=T * D * (SIZE[c["x"]] + outs) + 4 * outs * (T * D // per + 1), flops=3 * T * D * outs)
    if c["op"] == "fp8":
        M, N, K = c["M"], c["N"], c["K"]
        scales = _blocks(K) * (M + (N if c["block"] == "row" else _blocks(N)))
        return dict(bytes=M * K + N * K + 4 * scales + M * N * SIZE[c["out"]] * (1 + c["add"]), flops=2 * M * N * K)
    T, D, F, E, k = c["T"], c["D"], c["F"], c["E"], c["k"]
    active = E * (1 - (1 - k / E) ** T)  # experts that some token chooses
    es = SIZE[c["x"]]
    experts = active * 3 * D * F * (SIZE[c["w"]] + (4 / BLOCK ** 2 if c["w"] == "e4m3" else 0))
    return dict(bytes=int(experts + E * D * es + 2 * T * D * es + T * k * 8),
                flops=int(2 * T * E * D + 6 * T * k * D * F))
