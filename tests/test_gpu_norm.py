"""The norms around a block, their gate and residual scale, and their gradients against 64 bits.

Bounds, derived before any run.  Every output is rounded once (u of its type).  A row's sums run over at most 32
columns in a thread, 5 steps in a warp and 32 warps: they are off by at most 2^-24 * 80 of their terms'
magnitudes; with a handful of products around them each fp32 result is off by at most EPS = 2^-24 * 256 of the
magnitudes that enter it.  Sums over rows add their number of terms per thread and per partial row.
"""
import pytest
import torch

from dense_gemm_elementwise_gb300 import build as gbuild

gbuild.build()
from dense_gemm_elementwise_gb300 import binding as B  # noqa: E402

TYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -130, "f32": 2.0 ** -130}
EPS = 2.0 ** -24 * 256
SENT = 55.0


def unit(v, kind, eps):
    """N(v), its inverse divisor, and the magnitude that its fp32 rounding goes by."""
    if kind == "none":
        return v, torch.ones_like(v[:, :1]), v.abs()
    mag = v.abs()
    if kind == "layer":
        m = v.mean(1, keepdim=True)
        mag = mag + v.abs().mean(1, keepdim=True)
        v = v - m
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    # the divisor's own error: the centring's, relative to the rows' spread
    return v * r, r, (mag + v.abs() * (mag * r).pow(2).mean(1, keepdim=True).sqrt()) * r


def unit_grad(d, u, r, kind):
    if kind == "none":
        return d
    out = d - u * (d * u).mean(1, keepdim=True)
    if kind == "layer":
        out = out - d.mean(1, keepdim=True)
    return out * r


class Case:
    def __init__(self, T, D, x="bf16", w="f32", pre="rms", post="rms", gate=0, alpha=0.75, pad=(0, 0, 0, 0), eps=(1e-5, 1e-3),
                 weights=True, block=True, seed=0, shift=0.5):
        gen = torch.Generator().manual_seed(seed + T * 7 + D)
        dev = torch.device("cuda", 0)
        self.T, self.D, self.x, self.w, self.pre, self.post, self.alpha, self.eps = T, D, x, w, pre, post, alpha, eps
        self.ld = [D + p for p in pad]
        self.rpg = gate
        self.groups = -(-T // gate) if gate else 0

        def rows(scale, ld, shift=0.0):
            buf = torch.full((T, ld), float("nan"), dtype=TYPE[x], device=dev)
            buf[:, :D] = (torch.randn(T, D, generator=gen) * scale + shift).to(dev)
            return buf[:, :D]

        def vec(*shape):
            return (1 + 0.3 * torch.randn(*shape, generator=gen)).to(TYPE[w]).to(dev)

        self.xs = rows(2.0, self.ld[0], shift)
        self.b = rows(1.5, self.ld[1], -shift) if block else None
        self.y = rows(2.0, self.ld[2], shift)
        self.dy, self.dh = rows(1.0, self.ld[2]), rows(1.0, self.ld[3])
        self.gate = vec(self.groups, D) if gate and block else None
        self.w_post = vec(D) if weights and block and post != "none" else None
        self.w_pre = vec(D) if weights else None
        self.desc = B.make_norm_desc(x, w, pre, post, eps[0], eps[1], alpha, gate, *self.ld)
        self.plan = B.gemm_epi_norm_plan_create(T, D, self.desc)
        self.made = []

    def out(self, ld, dtype=None, n=None):
        n = self.T if n is None else n
        buf = torch.full((n * ld + 32,), SENT, dtype=TYPE[dtype or self.x], device=self.xs.device)
        v = buf[16:-16].view(n, ld)[:, :self.D]
        self.made.append((buf, n, ld))
        return v

    def untouched(self):
        for buf, n, ld in self.made:
            assert bool((buf[:16] == SENT).all()) and bool((buf[-16:] == SENT).all())
            assert bool((buf[16:-16].view(n, ld)[:, self.D:] == SENT).all())

    def at(self):
        return torch.arange(self.T, device=self.xs.device) // self.rpg

    def branch(self, b):
        n, r, mag = unit(b, self.post, self.eps[1])
        f = torch.full_like(b, self.alpha)
        if self.w_post is not None:
            f = f * self.w_post.double()
        if self.gate is not None:
            f = f * self.gate.double()[self.at()]
        return n, r, mag, f

    def close(self, got, want, bound, t):
        off = (got.double() - want).abs()
        bound = bound + U[t] * want.abs() + TINY[t]
        assert bool((off <= bound).all()), float((off / bound).max())

    def forward(self, y=True, h=True):
        yo, ho = self.out(self.ld[2]) if y else None, self.out(self.ld[3]) if h else None
        B.gemm_epi_norm_run(self.plan, self.xs, self.b, self.gate, self.w_post, self.w_pre, yo, ho)
        return yo, ho

    def check_forward(self, yo, ho):
        torch.cuda.synchronize()
        self.untouched()
        x = self.xs.double()
        y, ymag = x, torch.zeros_like(x)
        if self.b is not None:
            n, r, mag, f = self.branch(self.b.double())
            y, ymag = x + f * n, EPS * (x.abs() + f.abs() * mag)
        if yo is not None:
            self.close(yo, y, ymag, self.x)
        if ho is not None:
            u, r, mag = unit(y, self.pre, self.eps[0])
            w = self.w_pre.double() if self.w_pre is not None else 1.0
            spread = ymag.pow(2).mean(1, keepdim=True).sqrt() + ymag
            self.close(ho, u * w, (EPS * mag + 2 * r * spread * (1 + u.abs())) * abs(w), self.x)

    def grads(self, dy=True, db=True, sums=True):
        o = dict(dx=self.out(self.ld[0]), db=self.out(self.ld[1]) if db and self.b is not None else None,
                 dgate=self.out(self.D, self.w, self.groups) if sums and self.gate is not None else None,
                 dw_post=self.out(self.D, self.w, 1) if sums and self.w_post is not None else None,
                 dw_pre=self.out(self.D, self.w, 1) if sums and self.w_pre is not None else None)
        ws = torch.full((B.gemm_epi_norm_workspace_bytes(self.plan),), 0xFF, dtype=torch.uint8, device=self.xs.device)
        B.gemm_epi_norm_grad(self.plan, self.dy if dy else None, self.dh, self.y, self.b, self.gate, self.w_post, self.w_pre,
                             o["dx"], o["db"], o["dgate"], o["dw_post"], o["dw_pre"], ws)
        return o

    def check_grads(self, o, dy=True):
        torch.cuda.synchronize()
        self.untouched()
        d, dh, y = (self.dy.double() if dy else torch.zeros_like(self.dh.double())), self.dh.double(), self.y.double()
        u, r, mag = unit(y, self.pre, self.eps[0])
        e = dh if self.w_pre is None else dh * self.w_pre.double()
        t = d + unit_grad(e, u, r, self.pre)
        em = (e * mag).abs()
        tb = EPS * (d.abs() + r * (e.abs() + mag * em.mean(1, keepdim=True) + (e.abs().mean(1, keepdim=True))) * (1 + mag.pow(2).mean(1, keepdim=True).sqrt()))
        self.close(o["dx"], t, tb, self.x)
        rows = EPS + 2.0 ** -24 * (self.T + 64)
        if o["dw_pre"] is not None:
            self.close(o["dw_pre"][0], (dh * u).sum(0), rows * (dh.abs() * mag).sum(0), self.w)
        if self.b is None:
            return
        n, rb, nmag, f = self.branch(self.b.double())
        fd = f * t
        db = unit_grad(fd, n, rb, self.post)
        fdb = f.abs() * (tb + EPS * t.abs())
        fm = ((fd.abs() + fdb) * nmag).mean(1, keepdim=True)
        dbb = EPS * rb * (fd.abs() + nmag * fm + fd.abs().mean(1, keepdim=True)) * (1 + nmag.pow(2).mean(1, keepdim=True).sqrt()) \
            + rb * (fdb + nmag * (fdb * nmag).mean(1, keepdim=True) + fdb.mean(1, keepdim=True))
        if o["db"] is not None:
            self.close(o["db"], db, dbb, self.x)
        q, qm = t * n, (t.abs() + tb) * nmag * rows + tb * nmag
        if o["dgate"] is not None:
            w = self.alpha * (self.w_post.double() if self.w_post is not None else 1.0)
            want = torch.zeros(self.groups, self.D, dtype=torch.float64, device=q.device).index_add_(0, self.at(), q * w)
            bound = torch.zeros_like(want).index_add_(0, self.at(), qm * abs(w))
            self.close(o["dgate"], want, bound, self.w)
        if o["dw_post"] is not None:
            g = self.alpha * (self.gate.double()[self.at()] if self.gate is not None else 1.0)
            self.close(o["dw_post"][0], (q * g).sum(0), (qm * abs(g)).sum(0) if torch.is_tensor(g) else qm.sum(0) * abs(g), self.w)


SIZES = [(1, 1), (1, 7), (1, 4096), (2, 8), (3, 64), (5, 257), (33, 1024), (64, 1000), (100, 2048), (7, 4100), (1000, 96), (2500, 40),
         (19, 5120), (9, 8192), (5, 12345), (4, 16384), (3, 16383), (300, 10000)]


@pytest.mark.gpu
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,D", SIZES)
def test_forward_sizes(T, D, x):
    c = Case(T, D, x, gate=1 if T == 5 else T)
    c.check_forward(*c.forward())


@pytest.mark.gpu
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,D", SIZES)
def test_grad_sizes(T, D, x):
    c = Case(T, D, x, gate=1 if T == 5 else T)
    c.check_grads(c.grads())


# Rows of no whole 16-byte units, on both sides of each change of threads and columns per thread
@pytest.mark.gpu
@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("groups", ["one", "many"])
@pytest.mark.parametrize("T,D", [(3, 2), (700, 238), (40, 1030), (500, 4094), (460, 4098), (460, 4099), (9, 8190), (7, 8191), (9, 8194), (5, 16382)])
def test_other_widths(T, D, groups, x):
    c = Case(T, D, x, "bf16", "layer", "rms", T if groups == "one" else 2)
    c.check_forward(*c.forward())
    c.check_grads(c.grads())


# Odd widths with even pitches: rows end in half a pair
@pytest.mark.gpu
@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(3, 1), (4, 3), (700, 237), (301, 1803), (300, 4101), (9, 8189), (7, 8195), (5, 16383)])
def test_odd_widths_even_pitches(T, D, x):
    for gate in (0, 2):
        c = Case(T, D, x, "bf16", "layer", "rms", gate, pad=(1, 3, 1, 5))
        c.check_forward(*c.forward())
        c.check_grads(c.grads())


# Gate groups cut up, put together and over the edges of CTAs' runs of rows, in several waves of CTAs or one
@pytest.mark.gpu
@pytest.mark.parametrize("T,D,gate", [(4001, 1100, 12), (4001, 1101, 12), (1999, 4096, 5), (1999, 4096, 8), (5000, 520, 40), (5000, 520, 57), (900, 2056, 899),
                                      (900, 9000, 3), (20000, 24, 70), (20000, 24, 1)])
def test_gate_groups(T, D, gate):
    c = Case(T, D, "bf16", "f32", "rms", "rms", gate)
    c.check_forward(*c.forward())
    c.check_grads(c.grads())


KINDS = [("rms", "none"), ("rms", "rms"), ("layer", "none"), ("layer", "layer"), ("rms", "layer"), ("layer", "rms")]


@pytest.mark.gpu
@pytest.mark.parametrize("w", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pre,post", KINDS)
@pytest.mark.parametrize("T,D,gate", [(70, 130, 0), (70, 136, 70), (70, 200, 1), (71, 200, 9), (700, 64, 200)])
def test_kinds(T, D, gate, pre, post, w):
    c = Case(T, D, "f32", w, pre, post, gate, shift=1.0)
    c.check_forward(*c.forward())
    c.check_grads(c.grads())


@pytest.mark.gpu
@pytest.mark.parametrize("T,gate", [(3000, 1), (3000, 2), (3000, 7), (3000, 100), (3000, 1000), (3001, 1500), (3000, 2999), (3000, 9999)])
def test_gates_of_every_length(T, gate):
    c = Case(T, 72, "bf16", "f32", "rms", "rms", gate)
    c.check_forward(*c.forward())
    c.check_grads(c.grads())


@pytest.mark.gpu
@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [(8, 16, 24, 32), (1, 2, 3, 5), (0, 1, 0, 0)])
@pytest.mark.parametrize("D", [128, 77])
def test_pitches(D, pad, x):
    c = Case(37, D, x, "bf16", pad=pad, gate=10)
    c.check_forward(*c.forward())
    c.check_grads(c.grads())


@pytest.mark.gpu
def test_parts_left_out():
    c = Case(50, 256, block=False)
    c.check_forward(*c.forward())
    c.check_forward(*c.forward(y=False))
    c.check_grads(c.grads())
    c = Case(50, 256, weights=False, gate=5)
    c.check_forward(*c.forward(h=False))
    c.check_grads(c.grads(dy=False), dy=False)
    c = Case(50, 256, gate=5)
    c.check_grads(c.grads(db=False, sums=False))


@pytest.mark.gpu
def test_rows_of_zeros_and_of_equal_values():
    c = Case(40, 128, "f32", pre="layer", post="layer", shift=0.0)
    c.xs[::3] = 0
    c.b[::2] = 0
    c.b[1::4] = 3.0  # centred: nothing left but eps
    c.y[::5] = 0
    c.check_forward(*c.forward())
    c.check_grads(c.grads())


@pytest.mark.gpu
def test_nan_and_infinity_stay_in_their_rows():
    c = Case(64, 512, gate=8)
    c.b[3, 5] = float("nan")
    c.xs[10, 0] = float("inf")
    y, h = c.forward()
    torch.cuda.synchronize()
    bad = torch.zeros(64, dtype=torch.bool, device=y.device)
    bad[[3, 10]] = True
    assert bool(torch.isfinite(h[~bad]).all()) and bool(torch.isnan(h[bad]).any(1).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T,D", [(50, 256), (50, 999)])
def test_in_place(T, D):
    c = Case(T, D, gate=7)
    y, h = c.forward()
    x, b = c.xs.clone(), c.b.clone()
    B.gemm_epi_norm_run(c.plan, x, b, c.gate, c.w_post, c.w_pre, x, b)
    torch.cuda.synchronize()
    assert torch.equal(x, y) and torch.equal(b, h)
    o = c.grads()
    dy, b = c.dy.clone(), c.b.clone()
    ws = torch.empty(B.gemm_epi_norm_workspace_bytes(c.plan), dtype=torch.uint8, device=b.device)
    B.gemm_epi_norm_grad(c.plan, dy, c.dh, c.y, b, c.gate, c.w_post, c.w_pre, dy, b, None, None, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(dy, o["dx"]) and torch.equal(b, o["db"])


# outputs in every place that may be theirs, however rows are moved: whole 16-byte units, read when wanted above 8192
# columns, pairs and single elements, with and without a ring
@pytest.mark.gpu
@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("D", [12, 1026, 1111, 5000, 5001, 5002, 9000, 9001, 9002, 16384])
def test_in_place_whatever_the_width(D, x):
    c = Case(90, D, x, "bf16", "layer", "rms", 7)
    want = c.forward()
    c.check_forward(*want)
    for places in ("xb", "bx", "x-", "-b", "b-", "-x"):
        at = dict(x=c.xs.clone(), b=c.b.clone())
        y, h = (at.get(k, None) if k != "-" else c.out(D) for k in places)
        B.gemm_epi_norm_run(c.plan, at["x"], at["b"], c.gate, c.w_post, c.w_pre, y, h)
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(h, want[1]), places
    o = c.grads()
    c.check_grads(o)
    ws = torch.empty(B.gemm_epi_norm_workspace_bytes(c.plan), dtype=torch.uint8, device=c.b.device)
    for dx, db in (("dy", "b"), ("dy", "dh"), ("dh", "b"), ("y", "dy"), ("b", "y")):
        at = dict(dy=c.dy.clone(), dh=c.dh.clone(), y=c.y.clone(), b=c.b.clone())
        B.gemm_epi_norm_grad(c.plan, at["dy"], at["dh"], at["y"], at["b"], c.gate, c.w_post, c.w_pre, at[dx], at[db], None, None, None, ws)
        torch.cuda.synchronize()
        assert torch.equal(at[dx], o["dx"]) and torch.equal(at[db], o["db"]), (dx, db)


@pytest.mark.gpu
def test_another_stream_a_graph_and_the_same_bits():
    c = Case(500, 320, gate=100)
    a, b = c.grads(), c.grads()
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]), k
    y, h = c.forward()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, h2 = c.out(c.ld[2]), c.out(c.ld[3])
    B.gemm_epi_norm_run(c.plan, c.xs, c.b, c.gate, c.w_post, c.w_pre, y2, h2, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert B.prepare_norm_run(c.plan, c.xs, c.b, c.gate, c.w_post, c.w_pre, y2, h2)() == B.GE_OK
    c.xs.mul_(0.5)
    graph.replay()
    c.check_forward(y2, h2)


# rows per batch, the wider and the narrower rows of two plans that share kernels
@pytest.mark.gpu
@pytest.mark.parametrize("T,wide,narrow,x", [(700, 4096, 2560, "bf16"), (5, 4096, 320, "bf16"), (40, 4094, 1026, "f32"), (40, 4001, 1001, "f32"),
                                             (40, 4001, 301, "f16"), (9, 16384, 9000, "f16"), (9, 16382, 9002, "bf16"), (9, 16383, 9001, "f16")])
def test_a_plan_outlives_the_making_of_smaller_ones(T, wide, narrow, x):
    c = [Case(T, D, x, gate=2) for D in (wide, narrow)]
    for k in c:
        k.check_forward(*k.forward())
        k.check_grads(k.grads())


@pytest.mark.gpu
def test_offsets_past_32_bits():
    T, D = 140000, 16384
    dev = torch.device("cuda", 0)
    x = torch.zeros(T, D, dtype=torch.bfloat16, device=dev)
    x[-1] = 2.0
    plan = B.gemm_epi_norm_plan_create(T, D, B.make_norm_desc("bf16", "f32", eps_pre=0.25))
    h = torch.empty_like(x)
    B.gemm_epi_norm_run(plan, x, None, None, None, None, None, h)
    torch.cuda.synchronize()
    assert bool((h[-1].float() == torch.tensor(2 / 4.25 ** 0.5).bfloat16().float().item()).all()) and float(h[:-1].abs().max()) == 0
    ws = torch.empty(B.gemm_epi_norm_workspace_bytes(plan), dtype=torch.uint8, device=dev)
    B.gemm_epi_norm_grad(plan, None, x, x, None, None, None, None, h, None, None, None, None, ws)
    torch.cuda.synchronize()
    # all columns equal: d = 2 r (1 - 4 r^2) with r^2 = 1 / 4.25
    want = 2 / 4.25 ** 0.5 * (1 - 4 / 4.25)
    assert abs(float(h[-1, -1]) - want) <= 2.0 ** -8 * want and float(h[:-1].abs().max()) == 0


@pytest.mark.parametrize("pre,post", KINDS)
def test_gradient_formula_against_differences(pre, post):
    gen = torch.Generator().manual_seed(1)
    T, D, eps, alpha = 3, 6, (1e-2, 2e-2), 0.6
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, b, gate, wp, wq, gy, gh = rnd(T, D), rnd(T, D), rnd(2, D), rnd(D), rnd(D), rnd(T, D), rnd(T, D)
    at = torch.tensor([0, 0, 1])

    def f(x, b, gate, wp, wq):
        y = x + alpha * gate[at] * unit(b, post, eps[1])[0] * wp
        return float((y * gy).sum() + (unit(y, pre, eps[0])[0] * wq * gh).sum())

    n, rb, _ = unit(b, post, eps[1])
    y = x + alpha * gate[at] * n * wp
    u, r, _ = unit(y, pre, eps[0])
    t = gy + unit_grad(gh * wq, u, r, pre)
    q = t * n
    want = [t, unit_grad(alpha * gate[at] * wp * t, n, rb, post), torch.zeros(2, D, dtype=torch.float64).index_add_(0, at, alpha * wp * q),
            alpha * (gate[at] * q).sum(0), (gh * u).sum(0)]
    args = [x, b, gate, wp, wq]
    h = 1e-5
    for k, v in enumerate(args):
        flat = want[k].reshape(-1)
        for i in range(v.numel()):
            e = torch.zeros(v.numel(), dtype=torch.float64)
            e[i] = h
            up, dn = list(args), list(args)
            up[k], dn[k] = v + e.view_as(v), v - e.view_as(v)
            assert abs((f(*up) - f(*dn)) / (2 * h) - float(flat[i])) < 1e-7


@pytest.mark.gpu
def test_in_place_of_another_pitch_is_refused():
    c = Case(8, 64, pad=(0, 8, 16, 24))  # x, b, y, h
    big = lambda: torch.zeros(8 * 88, dtype=torch.bfloat16, device=c.xs.device)  # noqa: E731
    a = {k: big() for k in ("dy", "dh", "y", "b", "dx", "db")}
    ws = torch.empty(B.gemm_epi_norm_workspace_bytes(c.plan), dtype=torch.uint8, device=c.xs.device)

    def grad(**kw):
        p = {**a, **{k: a[v] for k, v in kw.items()}}
        return B.gemm_epi_norm_grad(c.plan, p["dy"], p["dh"], p["y"], p["b"], None, None, None, p["dx"], p["db"], None, None, None, ws, check=False)

    for k in ("dy", "dh", "y", "b"):
        assert grad(dx=k) == B.GE_ERR_INVALID, k
    for k in ("dy", "dh", "y"):
        assert grad(db=k) == B.GE_ERR_INVALID, k
    assert grad() == grad(db="b") == B.GE_OK
    torch.cuda.synchronize()


def _create(T=4, D=8, **kw):
    return B.gemm_epi_norm_plan_create(T, D, B.make_norm_desc(**{"x": "bf16", "w": "f32", **kw}))


@pytest.mark.parametrize("kw,status", [
    (dict(x=3), "UNSUPPORTED"), (dict(w=-1), "UNSUPPORTED"), (dict(pre="none"), "INVALID"), (dict(post=3), "INVALID"),
    (dict(eps_pre=-1.0), "INVALID"), (dict(eps_post=float("nan")), "INVALID"), (dict(alpha=float("inf")), "INVALID"),
    (dict(rows_per_gate=-1), "INVALID"), (dict(T=0), "SHAPE"), (dict(D=0), "SHAPE"), (dict(D=16385), "SHAPE"), (dict(T=1 << 31), "SHAPE"),
    (dict(ldx=7), "SHAPE")], ids=str)
def test_plan_refusals(kw, status):
    with pytest.raises(B.GemmEpiError) as e:
        _create(**kw)
    assert e.value.status == getattr(B, "GE_ERR_" + status)


def test_null_plans():
    assert B.lib.gemm_epi_norm_plan_create(None, 1, 1, None) == B.GE_ERR_INVALID
    assert B.gemm_epi_norm_workspace_bytes(None) == 0
    assert B.lib.gemm_epi_norm_run(None, *[None] * 8) == B.GE_ERR_INVALID
    B.gemm_epi_norm_plan_destroy(None)


@pytest.mark.gpu
def test_run_refusals():
    c = Case(8, 64, gate=2)
    y, h = c.out(64), c.out(64)

    def run(**kw):
        a = dict(x=c.xs, b=c.b, gate=c.gate, w_post=c.w_post, w_pre=c.w_pre, y=y, h=h, check=False)
        a.update(kw)
        return B.gemm_epi_norm_run(c.plan, **a)

    assert run(x=None) == run(gate=None) == run(y=None, h=None) == B.GE_ERR_MISSING_ARG
    assert run(b=None) == run(h=y) == B.GE_ERR_INVALID  # a gate without a block; two outputs in one place
    for k in ("x", "b", "y", "h", "gate"):
        p = dict(x=c.xs, b=c.b, y=y, h=h, gate=c.gate)[k].data_ptr()
        assert run(**{k: p + 2}) == B.GE_ERR_MISALIGNED, k
    dx, db, ws = c.out(64), c.out(64), torch.empty(B.gemm_epi_norm_workspace_bytes(c.plan), dtype=torch.uint8, device=y.device)

    def grad(**kw):
        a = dict(dy=c.dy, dh=c.dh, y=c.y, b=c.b, gate=c.gate, w_post=c.w_post, w_pre=c.w_pre, dx=dx, db=db, dgate=None, dw_post=None,
                 dw_pre=None, workspace=ws, check=False)
        a.update(kw)
        return B.gemm_epi_norm_grad(c.plan, **a)

    assert grad(dh=None) == grad(y=None) == grad(dx=None) == B.GE_ERR_MISSING_ARG
    assert grad(db=dx) == grad(w_pre=None, dw_pre=c.w_pre) == grad(b=None, gate=None, w_post=None) == B.GE_ERR_INVALID
    assert grad(workspace_bytes=ws.numel() - 1) == grad(workspace=None, workspace_bytes=1 << 20) == B.GE_ERR_WORKSPACE
    plain = Case(8, 64)
    assert B.gemm_epi_norm_run(plain.plan, plain.xs, plain.b, c.gate, None, None, y, h, check=False) == B.GE_ERR_INVALID
    assert run() == grad() == B.GE_OK
    torch.cuda.synchronize()
