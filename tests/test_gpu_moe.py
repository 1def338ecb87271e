"""A mixture-of-experts layer for a few tokens against 64 bits.

Bounds, derived before any run.  Weights and inputs are exact.  A sum of n products in fp32 whose additions may cut off is
off by at most n 2^-23 of its magnitudes (n: columns of a warp, joined by a few more); 8-bit weights' scales round once
more.  |act'| <= 1.13 for SiLU and GELU, so h = act(g) u is off by 1.13 |u| dg + |act(g)| du, and by the activation's own roundings,
2^-20, and by what two 16-bit values leave of it (2^-16).  y adds F products of each chosen expert, times weights that are off by
2^-20, and is rounded once (u).
"""
import pytest
import torch

from dense_gemm_elementwise_gb300 import build as gbuild

gbuild.build()
from dense_gemm_elementwise_gb300 import binding as B  # noqa: E402

TYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
        "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -130}
SENT = 33.0
ACT = {"silu": lambda v: v / (1 + (-v).exp()), "gelu": lambda v: v / 2 * torch.erfc(-v / 2 ** 0.5), "relu": lambda v: v.clamp_min(0)}


def blocks(n):
    return -(-n // 128)


class Case:
    def __init__(self, T, D, F, E, k, x="bf16", w=None, router=None, score="softmax", norm=True, bias=False, scale=1.0,
                 act="silu", pad=(0, 0), seed=0, **kw):
        w, router = w or x, router or x
        g = torch.Generator(device="cuda").manual_seed(seed + T * 7 + D * 3 + F + E)
        dev = torch.device("cuda", 0)
        randn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
        self.T, self.D, self.F, self.E, self.k, self.xt = T, D, F, E, k, x
        self.score, self.norm, self.scale, self.act = score, norm, scale, act
        self.x = torch.full((T, D + pad[0]), float("nan"), dtype=TYPE[x], device=dev)[:, :D]
        self.x.copy_(randn(T, D))
        self.router = (randn(E, D) * D ** -0.5).to(TYPE[router])
        self.bias = 0.2 * randn(E) if bias else None
        self.k8 = w in LARGEST
        self.w, self.s = {}, {}
        for name, rows, cols in (("up", 2 * F, D), ("down", D, F)):
            v = randn(E, rows, cols)
            self.s[name] = None
            if self.k8:
                self.w[name] = (v * (LARGEST[w] / 4)).clamp(-LARGEST[w], LARGEST[w]).to(TYPE[w])
                self.s[name] = (0.5 + torch.rand(E, blocks(cols), blocks(rows), generator=g, device=dev)) * (4 / LARGEST[w] * cols ** -0.5)
            else:
                self.w[name] = (v * cols ** -0.5).to(TYPE[w])
        self.buf = torch.full((T + 2, D + pad[1]), SENT, dtype=TYPE[x], device=dev)
        self.index = torch.full((T + 1, k), -5, dtype=torch.int32, device=dev)
        self.weight = torch.full((T + 1, k), SENT, device=dev)
        self.desc = B.make_moe_desc(x, w, router, score=score, renormalise=norm, act=act, route_scale=scale, ldx=D + pad[0],
                                    ldy=D + pad[1], **kw)
        self.plan = B.gemm_epi_moe_plan_create(T, D, F, E, k, self.desc)
        self.ws = torch.full((B.gemm_epi_moe_workspace_bytes(self.plan),), 0xFF, dtype=torch.uint8, device=dev)

    def run(self, stream=None, index=True, weight=True):
        B.gemm_epi_moe_run(self.plan, self.x, self.router, self.bias, self.w["up"], self.s["up"], self.w["down"], self.s["down"],
                           self.buf, self.index if index else None, self.weight if weight else None, self.ws, stream=stream)
        return self

    def weights(self, name, e):
        w = self.w[name][e].double()
        if self.s[name] is not None:
            s = self.s[name][e].double().t()
            w = w * s.repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :w.shape[1]]
        return w

    def routing(self):
        logits = self.x.double() @ self.router.double().t()
        p = torch.softmax(logits, 1) if self.score == "softmax" else 1 / (1 + (-logits).exp())
        by = logits if self.bias is None else p + self.bias.double()
        index = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :self.k]
        weight = p.gather(1, index)
        if self.norm:
            weight = weight / weight.sum(1, keepdim=True)
        return index, weight * self.scale

    def want(self, index, weight):
        x = self.x.double()
        y, lim = torch.zeros_like(x), torch.zeros_like(x)
        fd, ff = (self.D + 16) * 2.0 ** -23, (self.F + 16) * 2.0 ** -23
        for e in range(self.E):
            t, j = (index == e).nonzero(as_tuple=True)
            if not t.numel():
                continue
            up, down = self.weights("up", e), self.weights("down", e)
            g, u = (x[t] @ up.t()).split(self.F, 1)
            dg, du = (x[t].abs() @ up.abs().t() * fd).split(self.F, 1)
            a = ACT[self.act](g)
            h = a * u
            dh = 1.13 * u.abs() * dg + a.abs() * du + h.abs() * (2.0 ** -20 + 2.0 ** -16) + TINY[self.xt]
            wt = weight[t, j][:, None]
            y.index_add_(0, t, (h @ down.t()) * wt)
            lim.index_add_(0, t, (dh @ down.abs().t() + (h.abs() @ down.abs().t()) * (ff + 2.0 ** -20)) * wt.abs())
        return y, lim

    def check(self, index=True, weight=True, rows=None, close=True):
        torch.cuda.synchronize()
        assert B.gemm_epi_last_error() == B.GE_OK
        T = self.T
        rows = torch.arange(T, device=self.x.device) if rows is None else rows
        wi, ww = self.routing()
        if index:
            assert torch.equal(self.index[rows].long(), wi[rows]), (self.index[rows].long() != wi[rows]).nonzero()[:5]
            assert bool((self.index[T:] == -5).all())
        else:
            assert bool((self.index == -5).all())
        if weight:
            assert bool(((self.weight[rows].double() - ww[rows]).abs() <= 2.0 ** -20 * ww[rows].abs()).all())
            assert bool((self.weight[T:] == SENT).all())
        y, lim = self.want(wi, ww)
        got = self.buf[:T, :self.D]
        off, lim = (got.double() - y).abs()[rows], (lim * (1 + U[self.xt]) + y.abs() * U[self.xt] + TINY[self.xt])[rows]
        assert bool((off <= lim).all()), ((off / lim).max().item(), (~(off <= lim)).nonzero()[:4].tolist())
        assert bool((self.buf[T:] == SENT).all()) and bool((self.buf[:, self.D:] == SENT).all())
        if close:
            B.gemm_epi_moe_plan_destroy(self.plan)


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,F,E,k", [(1, 8, 8, 1, 1), (1, 256, 128, 8, 2), (2, 1024, 136, 4, 4), (3, 1000, 520, 13, 3), (8, 512, 256, 16, 2),
                                       (9, 264, 72, 5, 2), (17, 128, 128, 3, 1), (40, 520, 264, 7, 5), (64, 256, 256, 33, 8),
                                       (128, 72, 40, 6, 2), (128, 136, 80, 300, 16), (5, 2056, 1032, 6, 2)])
@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_sizes(T, D, F, E, k, x):
    Case(T, D, F, E, k, x).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["e4m3", "e5m2"])
@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("T,D,F,E,k", [(1, 16, 16, 2, 1), (1, 512, 256, 8, 2), (6, 1008, 400, 9, 3), (30, 272, 144, 4, 2), (50, 400, 1040, 3, 2),
                                       (128, 256, 128, 2, 1)])
def test_weights_of_8_bits(T, D, F, E, k, x, w):
    Case(T, D, F, E, k, x, w).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("router", ["f32", "bf16"])
def test_routing(score, norm, bias, router):
    Case(37, 520, 64, 41, 6, score=score, norm=norm, bias=bias, router=router, scale=2.5).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_activations(act):
    Case(11, 256, 264, 4, 2, "f16", act=act).run().check()


@pytest.mark.gpu
def test_pitches_and_outputs_left_out():
    Case(7, 264, 64, 5, 2, pad=(8, 24)).run(index=False).check(index=False)
    c = Case(7, 264, 64, 5, 2, pad=(16, 0)).run(weight=False)
    c.check(weight=False)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [8, 9, 33, 128])
def test_all_tokens_choose_the_same_experts(T):
    c = Case(T, 256, 128, 20, 2)
    c.x.copy_(c.x[:1].expand(T, -1) * (1 + torch.arange(T, device=c.x.device)[:, None] / T))
    c.run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(bias, score):
    c = Case(20, 256, 64, 70, 8, score=score, bias=bias)
    c.router[35:] = c.router[:35]
    if bias:
        c.bias[35:] = c.bias[:35]
    c.run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("router", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(), dict(bias=True), dict(bias=True, score="sigmoid")])
def test_choices_between_logits_that_fp32_does_not_tell_apart(kw, router):
    """Pairs of experts whose logits, of several hundred terms, differ by one small product."""
    c = Case(16, 2048, 64, 64, 8, router=router, **kw)
    c.router[32:] = c.router[:32]
    c.router[32:, 5] += (2.0 ** -24 if router == "f32" else 2.0 ** -12) * (1 - 2 * (torch.arange(32, device=c.x.device) % 2))
    c.router[:, 6:12] *= 50.0  # large terms around it
    if c.bias is not None:
        c.bias[32:] = c.bias[:32]
    c.run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("score,bias", [("sigmoid", False), ("sigmoid", True), ("softmax", True)])
def test_scores_too_small_for_fp32_are_weighed_against_each_other(score, bias):
    c = Case(6, 64, 64, 41, 5, score=score, bias=bias)
    e = torch.arange(41, device=c.x.device)
    c.x.zero_()
    c.x[:, 0] = 1.0
    c.router.zero_()
    c.router[:, 0] = -(100.0 + e) if score == "sigmoid" else -4.0 * e
    if bias:
        c.bias.copy_(2.0 * e)
    c.run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("E,k", [(31, 5), (32, 16), (33, 1), (128, 16), (129, 16), (512, 16), (511, 3)])
@pytest.mark.parametrize("kw", [dict(), dict(bias=True, score="sigmoid"), dict(bias=True)])
def test_numbers_of_experts(E, k, kw):
    Case(19, 128, 16, E, k, **kw).run().check()


@pytest.mark.gpu
def test_large_logits():
    for score in ("softmax", "sigmoid"):
        c = Case(9, 256, 64, 10, 3, score=score, norm=False)
        c.router *= 20.0
        c.run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", True)])
@pytest.mark.parametrize("w", ["bf16", "e4m3"])
def test_nan_and_infinity_stay_in_their_tokens(score, bias, w):
    c = Case(20, 256, 128, 6, 2, w=w, score=score, bias=bias)
    c.x[3, 7] = float("nan")
    c.x[11, 9] = float("inf")
    c.run()
    torch.cuda.synchronize()
    assert bool(c.buf[3, :256].isnan().all())
    assert not bool(c.buf[11, :256].isfinite().any())
    at = c.index[:20]
    assert bool(((at >= 0) & (at < 6)).all()) and bool((at[:, 0] != at[:, 1]).all())
    rows = torch.tensor([i for i in range(20) if i not in (3, 11)], device=c.x.device)
    c.x[3] = c.x[11] = 0.0  # for the reference
    c.check(rows=rows)


@pytest.mark.gpu
def test_an_expert_of_nan_reaches_those_who_chose_it():
    c = Case(12, 256, 128, 6, 2)
    c.w["down"][2, 100] = float("nan")
    c.run()
    torch.cuda.synchronize()
    hit = (c.routing()[0] == 2).any(1)
    assert torch.equal(c.buf[:12, 100].isnan(), hit)
    assert not bool(c.buf[:12, :100].isnan().any()) and not bool(c.buf[:12, 101:].isnan().any())


@pytest.mark.gpu
@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("w,code", [("e4m3", 0x7F), ("e4m3", 0xFF), ("e5m2", 0x7C), ("e5m2", 0xFE)])
def test_weights_of_8_bits_that_are_no_numbers(x, w, code):
    """A row of w_down, and of gate or up, through which it reaches all of y; no other code counts as one."""
    for name, row in (("down", 100), ("up", 37), ("up", 128 + 90)):
        c = Case(12, 256, 128, 6, 2, x, w)
        c.w[name].view(torch.uint8)[2, row, 77] = code
        c.run()
        torch.cuda.synchronize()
        hit = (c.routing()[0] == 2).any(1)
        nan = c.buf[:12, :256].isnan()
        if name == "down":
            assert torch.equal(nan[:, 100], hit)
            nan[:, 100] = False
            assert not bool(nan.any())
        else:
            assert torch.equal(nan.all(1), hit) and torch.equal(nan.any(1), hit)
        B.gemm_epi_moe_plan_destroy(c.plan)


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["e4m3", "e5m2"])
@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_every_8_bit_value(x, w):
    """All finite codes, subnormals among them, in both products."""
    c = Case(5, 512, 256, 3, 2, x, w)
    codes = torch.arange(256, dtype=torch.uint8, device=c.x.device)
    codes = codes[codes.view(TYPE[w]).float().isfinite()]
    for name in ("up", "down"):
        v = c.w[name].view(torch.uint8)
        v.copy_(codes[torch.arange(v.numel(), device=v.device) * 7 % codes.numel()].view(v.shape))
        c.s[name].mul_(2.0 ** -3)
    c.run().check()


@pytest.mark.gpu
def test_weights_from_the_quantiser():
    """A layer whose experts gemm_epi_quant_run has quantised, against 64 bits of what the values stand for and, in the
    2-norm, of the weights themselves: three products with roundings of 2^-4 at most, independent for each weight."""
    c, d = Case(9, 400, 272, 5, 2), Case(9, 400, 272, 5, 2, w="e4m3")
    for name in ("up", "down"):
        for e in range(5):
            w = c.w[name][e].contiguous()
            rows, cols = w.shape
            plan = B.gemm_epi_quant_plan_create(rows, cols, B.make_quant_desc("bf16", "e4m3", block="square"))
            s = torch.empty(blocks(cols), blocks(rows), device=w.device)
            B.gemm_epi_quant_run(plan, w, d.w[name][e], s)
            torch.cuda.synchronize()
            d.s[name][e] = s
            B.gemm_epi_quant_plan_destroy(plan)
    for k in ("x", "router"):
        getattr(d, k).copy_(getattr(c, k))
    c.run().check()
    d.run().check()
    a, b = c.buf[:9, :400].double(), d.buf[:9, :400].double()
    assert float((a - b).norm() / a.norm()) <= 3 * 2.0 ** -4


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [10, 40])
def test_another_stream_a_graph_and_the_same_bits(T, w):
    c = Case(T, 512, 256, 12, 3, w=w, score="sigmoid", bias=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    torch.cuda.synchronize()
    first = c.buf.clone(), c.index.clone(), c.weight.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(stream=torch.cuda.current_stream())
        c.run(stream=torch.cuda.current_stream())
    for fill in (0x00, 0xFF, 0x55):
        c.buf.fill_(SENT)
        c.ws.fill_(fill)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, (c.buf, c.index, c.weight)):
            assert torch.equal(a, b)
    c.x.copy_(torch.flip(c.x, [0]))  # another input, in place
    graph.replay()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("k,D", [(2, 72), (16, 1000)])
def test_many_columns_of_y_at_once(k, D):
    """Units of one column of k: the shares of many columns become complete faster than they are added."""
    Case(128, D, 8, 16, k).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,D,F,E,k", [(1, 32, 16, 1, 1), (1, 96, 48, 2, 1), (2, 4096, 16, 3, 2), (5, 32, 512, 4, 2)])
def test_a_cta_with_units_that_wait_for_its_own(T, D, F, E, k, w):
    """Few units: a CTA takes some of h together with those that wait for it, in every mixture that comes up."""
    c = Case(T, D, F, E, k, w=w)
    for _ in range(200):
        c.run()
    c.check()


@pytest.mark.gpu
def test_two_at_once():
    """Two layers on two streams, each with its own workspace, more work than the GPU holds at a time."""
    cs = [Case(64, 1024, 512, 40, 4, seed=i) for i in range(2)]
    ss = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cs, ss):
            c.run(stream=s)
    for c in cs:
        c.check()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Weights of 2.4e9 elements, whose last experts alone are chosen."""
    E, D, F = 60, 4096, 3264
    c = Case(2, 64, 64, 4, 2)
    dev = torch.device("cuda", 0)
    up, down = torch.zeros(E, 2 * F, D, dtype=torch.bfloat16, device=dev), torch.zeros(E, D, F, dtype=torch.bfloat16, device=dev)
    up[-4:, :64, :64], up[-4:, F:F + 64, :64], down[-4:, :64, :64] = c.w["up"][:, :64], c.w["up"][:, 64:], c.w["down"]
    router = torch.zeros(E, D, dtype=torch.bfloat16, device=dev)
    router[-4:, :64] = c.router
    bias = torch.full((E,), -100.0, device=dev)
    bias[-4:] = 0.0
    x = torch.zeros(2, D, dtype=torch.bfloat16, device=dev)
    x[:, :64] = c.x
    c.bias = torch.zeros(4, device=dev)
    plan = B.gemm_epi_moe_plan_create(2, D, F, E, 2, B.make_moe_desc("bf16", "bf16", "bf16", score="sigmoid"))
    c.score = "sigmoid"
    y, index = torch.empty(2, D, dtype=torch.bfloat16, device=dev), torch.empty(2, 2, dtype=torch.int32, device=dev)
    ws = torch.empty(B.gemm_epi_moe_workspace_bytes(plan), dtype=torch.uint8, device=dev)
    B.gemm_epi_moe_run(plan, x, router, bias, up, None, down, None, y, index, None, ws)
    torch.cuda.synchronize()
    B.gemm_epi_moe_plan_destroy(plan)
    assert not bool(y[:, 64:].any())
    c.buf[:2, :64] = y[:, :64]
    c.index[:2] = index - (E - 4)
    c.check(weight=False)


@pytest.mark.gpu
def test_a_unit_that_never_comes_is_reported():
    c = Case(4, 256, 128, 4, 2, timeout_ms=50, debug_flags=B.GE_DEBUG_SKIP_FIRST_LOAD).run()
    torch.cuda.synchronize()
    assert B.gemm_epi_last_error() == B.GE_ERR_TIMEOUT
    B.gemm_epi_moe_plan_destroy(c.plan)
    Case(4, 256, 128, 4, 2).run().check()


def bad(T=4, D=64, F=64, E=8, k=2, x="bf16", w="bf16", router="bf16", **kw):
    reserved = kw.pop("reserved", 0)
    d = B.make_moe_desc(x, w, router, **kw)
    d.reserved = reserved
    with pytest.raises(B.GemmEpiError) as e:
        B.gemm_epi_moe_plan_create(T, D, F, E, k, d)
    return e.value.status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), "GE_ERR_SHAPE"), (dict(T=129), "GE_ERR_SHAPE"), (dict(E=513), "GE_ERR_SHAPE"), (dict(k=9), "GE_ERR_SHAPE"), (dict(k=0), "GE_ERR_SHAPE"),
    (dict(E=100, k=17), "GE_ERR_SHAPE"), (dict(D=0), "GE_ERR_SHAPE"), (dict(F=1 << 21), "GE_ERR_SHAPE"), (dict(x="f32"), "GE_ERR_UNSUPPORTED"),
    (dict(w="f16"), "GE_ERR_UNSUPPORTED"), (dict(router="f16"), "GE_ERR_UNSUPPORTED"), (dict(act="tanh"), "GE_ERR_UNSUPPORTED"),
    (dict(score=2), "GE_ERR_INVALID"), (dict(renormalise=2), "GE_ERR_INVALID"), (dict(timeout_ms=-1), "GE_ERR_INVALID"),
    (dict(debug_flags=2), "GE_ERR_INVALID"), (dict(route_scale=float("inf")), "GE_ERR_INVALID"), (dict(reserved=1), "GE_ERR_INVALID"),
    (dict(D=60), "GE_ERR_MISALIGNED"), (dict(F=68), "GE_ERR_MISALIGNED"), (dict(w="e4m3", F=72), "GE_ERR_MISALIGNED"),
    (dict(ldx=68), "GE_ERR_MISALIGNED"), (dict(ldy=56), "GE_ERR_SHAPE")])
def test_plan_refusals(kw, status):
    assert bad(**kw) == getattr(B, status)


def test_null_plans():
    assert B.lib.gemm_epi_moe_plan_create(None, 1, 8, 8, 1, 1, None) == B.GE_ERR_INVALID
    assert B.lib.gemm_epi_moe_run(*[None] * 12, 0, None) == B.GE_ERR_INVALID
    assert B.gemm_epi_moe_workspace_bytes(None) == 0
    B.gemm_epi_moe_plan_destroy(None)


@pytest.mark.gpu
def test_run_refusals():
    c, e = Case(4, 64, 64, 4, 2), Case(4, 64, 64, 4, 2, w="e4m3")

    def run(c, n=None, **kw):
        a = dict(x=c.x, w_router=c.router, bias=None, w_gate_up=c.w["up"], s_gate_up=c.s["up"], w_down=c.w["down"], s_down=c.s["down"],
                 y=c.buf, index=None, weight=None, workspace=c.ws)
        a.update(kw)
        return B.gemm_epi_moe_run(c.plan, workspace_bytes=c.ws.numel() if n is None else n, check=False, **a)

    for name in ("x", "w_router", "w_gate_up", "w_down", "y"):
        assert run(c, **{name: None}) == B.GE_ERR_MISSING_ARG
        assert run(c, **{name: c.ws.data_ptr() + 8}) == B.GE_ERR_MISALIGNED
    assert run(e, s_down=None) == B.GE_ERR_MISSING_ARG
    assert run(c, s_down=e.s["down"]) == B.GE_ERR_INVALID
    assert run(c, workspace=None) == B.GE_ERR_WORKSPACE
    assert run(c, n=c.ws.numel() - 1) == B.GE_ERR_WORKSPACE
    assert run(c, workspace=c.ws.data_ptr() + 8) == B.GE_ERR_MISALIGNED


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_weights_of_far_logits(score, bias, norm, T):
    """Logits up to 80 apart, each of 24 bits and more: weights from 1 to 1e-35 are within 2^-20 of themselves."""
    c = Case(T, 64, 16, 41, 16, score=score, bias=bias, norm=norm, router="f32")
    g = torch.Generator().manual_seed(2)
    c.x.zero_()
    c.x[:, 0] = 1 + torch.arange(T, device=c.x.device) % 8 / 32
    c.router.zero_()
    c.router[:, 0] = (-65 * torch.rand(41, generator=g)).to(c.x.device)
    c.run().check()


SCORES = [dict(), dict(norm=False), dict(score="sigmoid"), dict(bias=True), dict(bias=True, score="sigmoid")]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("E,k", [(2, 1), (7, 1), (32, 1), (33, 1), (64, 1), (70, 1), (32, 2), (40, 3), (64, 15), (64, 16), (128, 3)])
@pytest.mark.parametrize("kw", SCORES)
def test_equal_logits_of_all_experts(E, k, T, kw):
    """Tokens of zeros between others, and equal biases: the first k experts, in both places where a choice is made."""
    c = Case(T, 64, 16, E, k, **kw)
    c.x[::2] = 0.0
    if c.bias is not None:
        c.bias.fill_(0.125)
    c.run().check()
    assert bool((c.index[:T:2] == torch.arange(k, device=c.x.device)).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("E,k", [(4, 1), (4, 3), (32, 1), (32, 7), (40, 5), (64, 1), (64, 3), (64, 15), (128, 7)])
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("kw", SCORES)
def test_a_last_place_between_two_equal_experts(E, k, T, apart, kw):
    """Every expert is there twice, next to itself or half of all experts away, and an odd number of them is chosen."""
    c = Case(T, 256, 16, E, k, **kw)
    half = E // 2
    copies, of = (slice(half, E), slice(0, half)) if apart else (slice(1, E, 2), slice(0, E, 2))
    c.router[copies] = c.router[of]
    if c.bias is not None:
        c.bias[copies] = c.bias[of]
    c.run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("E,k", [(32, 1), (32, 5), (64, 1), (64, 7), (64, 15), (128, 3)])
@pytest.mark.parametrize("kw", SCORES)
def test_a_last_place_between_logits_that_fp32_does_not_tell_apart(E, k, T, kw):
    """As test_choices_between_logits_that_fp32_does_not_tell_apart, with an odd number chosen."""
    c = Case(T, 2048, 16, E, k, **kw)
    half = E // 2
    c.router[half:] = c.router[:half]
    c.router[half:, 5] += 2.0 ** -12 * (1 - 2 * (torch.arange(half, device=c.x.device) % 2))
    c.router[:, 6:12] *= 50.0
    if c.bias is not None:
        c.bias[half:] = c.bias[:half]
    c.run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("E,k", [(2, 1), (17, 1), (17, 4), (32, 3), (33, 1), (64, 1), (64, 5), (64, 16), (100, 3)])
def test_biased_scores_equal_in_fp32(E, k, T):
    """Sigmoids of 20 and more are 1 in fp32, and 1 - e^-l, 2e-9 and less below it, in 64 bits.  Logits are exact."""
    c = Case(T, 64, 16, E, k, score="sigmoid", bias=True, router="f32")
    g = torch.Generator().manual_seed(E)
    c.x[:, 0] = 1.0
    c.x[:, 1:] = 0.0
    c.router[:, 0] = (20.0 + torch.randperm(E, generator=g) / 32.0).to(c.x.device)
    c.bias.fill_(0.25)
    c.run().check()
    c = Case(T, 64, 16, E, k, score="sigmoid", bias=True, router="f32")  # (and some that 64 bits do not tell apart either)
    c.x[:, 0] = 1.0
    c.x[:, 1:] = 0.0
    c.router[:, 0] = (20.0 + torch.randperm(E, generator=g) // 2 / 32.0).to(c.x.device)
    c.bias.fill_(0.25)
    c.run().check()


@pytest.mark.parametrize("kw", [dict(ldx=1 << 31), dict(ldy=1 << 31), dict(D=(1 << 20) + 16)])
def test_largest_pitches_and_widths(kw):
    assert bad(**kw) == B.GE_ERR_SHAPE
