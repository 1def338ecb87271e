"""Vocabulary loss and its gradients against a 64-bit implementation of the formulas.

Bounds, all derived before any run.  Products of two 16-bit numbers are exact in fp32; a sum of n of them in the
tensor unit's groups of 16 is off by at most (n / 16 + 16) 2^-23 of the sum of their magnitudes (`acc`).  A logit is
then off by `acc` of |H| |W|^T; lse by that and the rounding of a handful of fp32 operations, 2^-20 (1 + |lse|);
p = exp(l - lse) is off by the sum of both, relatively.  dl is rounded once (u = 2^-8 for bf16, 2^-11 for f16), the
sums of the gradient products are off as above, and the results are rounded once more.
"""
import numpy as np
import pytest
import torch

from dense_gemm_elementwise_gb300 import build as gbuild

gbuild.build()
from dense_gemm_elementwise_gb300 import binding as B  # noqa: E402

TYPE = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
PAD = 1 << 7


def acc(n):
    return (n / 16 + 16) * 2.0 ** -23


def reference(H, W, target, weight, c, z, mean, g):
    """loss, lse, total, dH, dW, and the magnitudes that the bounds need; 64 bits, rows that take part only."""
    T, V = H.shape[0], W.shape[0]
    keep = ((target >= 0) & (target < V)).nonzero()[:, 0]
    Hd, Wd = H.double()[keep], W.double()
    w = (torch.ones(T, dtype=torch.float64, device=H.device) if weight is None else weight.double())[keep]
    r = torch.arange(keep.numel(), device=H.device)
    l = c * Hd @ Wd.T
    lse = torch.logsumexp(l, 1) if keep.numel() else torch.zeros(0, dtype=torch.float64, device=H.device)
    rows = w * (lse - l[r, target[keep]] + z * lse ** 2)
    norm = w.sum() if mean else torch.ones((), dtype=torch.float64, device=H.device)
    on = bool(norm != 0)
    total = rows.sum() / norm if on else torch.zeros((), dtype=torch.float64, device=H.device)
    p = torch.exp(l - lse[:, None])
    gw = w * g / norm if on else torch.zeros_like(w)
    zf = 1 + 2 * z * lse
    d = p * zf[:, None]
    d[r, target[keep]] -= 1
    d = d * gw[:, None]
    out = {"loss": torch.zeros(T, dtype=torch.float64, device=H.device), "lse": torch.zeros(T, dtype=torch.float64, device=H.device),
           "total": total, "dH": torch.zeros(T, H.shape[1], dtype=torch.float64, device=H.device), "dW": c * d.T @ Hd}
    out["loss"][keep], out["lse"][keep] = rows, lse
    out["dH"][keep] = c * d @ Wd
    return out, dict(keep=keep, Hd=Hd, Wd=Wd, w=w, p=p * (zf * gw).abs()[:, None], d=d.abs(), lse=lse, gw=gw.abs(), zf=zf.abs(),
                     mag=c * Hd.abs() @ Wd.abs().T if keep.numel() else torch.zeros(0, V, device=H.device))


class Case:
    def __init__(self, T, V, D, ab="bf16", index="i64", pad=(0, 0, 0, 0), c=1.0, z=0.0, mean=True, weights=None, ignored=0.0,
                 g=1.0, seed=0, buffer_bytes=0, scale=2.0, max_ctas=0):
        gen = torch.Generator().manual_seed(seed)
        dev = torch.device("cuda", 0)
        self.T, self.V, self.D, self.ab, self.c, self.z, self.mean, self.g = T, V, D, ab, c, z, mean, g
        self.ld = [-(-D // 8) * 8 + 8 * p for p in pad]
        dt = TYPE[ab]

        def wide(x, ld):
            buf = torch.full((x.shape[0], ld), float("nan"), dtype=dt, device=dev)  # what must not be read as data
            buf[:, :x.shape[1]] = x.to(dev)
            return buf[:, :x.shape[1]]

        self.H = wide(torch.randn(T, D, generator=gen), self.ld[0])
        self.W = wide(torch.randn(V, D, generator=gen) * (scale / D ** 0.5), self.ld[1])
        t = torch.randint(0, V, (T,), generator=gen)
        t[torch.rand(T, generator=gen) < ignored] = -100
        self.target = t.to(dev)
        self.weight = None
        if weights == "positive":
            self.weight = (torch.rand(T, generator=gen) + 0.5).to(dev)
        elif weights == "mixed":
            self.weight = (torch.randn(T, generator=gen) * (torch.rand(T, generator=gen) < 0.7)).to(dev)
        elif weights == "zero":
            self.weight = torch.zeros(T, device=dev)
        desc = B.make_xent_desc(ab, index, *self.ld, logit_scale=c, z_loss=z, reduction="mean" if mean else "sum",
                                buffer_bytes=buffer_bytes, max_ctas=max_ctas)
        self.index = index
        self.plan = B.gemm_epi_xent_plan_create(T, V, D, desc)

    def outputs(self):
        dev = self.H.device
        dt = TYPE[self.ab]
        self.buf = {k: torch.full((n * ld + 2 * PAD,), 77.0, dtype=dt, device=dev)
                    for k, n, ld in (("dH", self.T, self.ld[2]), ("dW", self.V, self.ld[3]))}
        o = {k: torch.full((n,), 77.0, device=dev) for k, n in (("loss", self.T), ("lse", self.T), ("total", 1))}
        for k, n, ld in (("dH", self.T, self.ld[2]), ("dW", self.V, self.ld[3])):
            o[k] = self.buf[k][PAD:-PAD].view(n, ld)[:, :self.D]
        return o

    def untouched(self):
        for k, n, ld in (("dH", self.T, self.ld[2]), ("dW", self.V, self.ld[3])):
            b = self.buf[k]
            assert bool((b[:PAD] == 77).all()) and bool((b[-PAD:] == 77).all()), k
            assert bool((b[PAD:-PAD].view(n, ld)[:, self.D:] == 77).all()), k

    def workspace(self, grads):
        return torch.full((B.gemm_epi_xent_workspace_bytes(self.plan, grads),), 0xFF, dtype=torch.uint8, device=self.H.device)

    def targets(self):
        return self.target.to(torch.int32) if self.index == "i32" else self.target

    def step(self, dH=True, dW=True, ws=None, stream=None):
        o = self.outputs()
        ws = self.workspace(True) if ws is None else ws
        B.gemm_epi_xent_step(self.plan, self.H, self.W, self.targets(), self.weight, self.g, o["loss"], o["lse"], o["total"],
                             o["dH"] if dH else None, o["dW"] if dW else None, ws, stream=stream)
        return o

    def loss(self):
        o = self.outputs()
        B.gemm_epi_xent_loss(self.plan, self.H, self.W, self.targets(), self.weight, o["loss"], o["lse"], o["total"], self.workspace(False))
        return o

    def check(self, o, grads=True, which=("dH", "dW")):
        torch.cuda.synchronize()
        assert B.gemm_epi_last_error() == B.GE_OK
        self.untouched()
        ref, m = reference(torch.nan_to_num(self.H) if self.clean else self.H, self.W, self.target, self.weight, self.c, self.z, self.mean, self.g)
        u = U[self.ab]
        c = abs(self.c)
        logit = acc(self.D) * (float(m["mag"].max()) if m["keep"].numel() else 0.0) * np.sign(self.c)
        logit = abs(logit) + 2.0 ** -22 * float((m["lse"].abs().max() if m["keep"].numel() else torch.zeros(())))
        lse = logit + 2.0 ** -20 * (1 + ref["lse"].abs())
        assert bool(((o["lse"].double() - ref["lse"]).abs() <= lse).all())
        w = torch.zeros_like(ref["loss"])
        w[m["keep"]] = m["w"].abs()
        row = w * (2 * lse + 2 * abs(self.z) * ref["lse"].abs() * lse) + 2.0 ** -23 * ref["loss"].abs()
        assert bool(((o["loss"].double() - ref["loss"]).abs() <= row).all())
        keep = ((self.target >= 0) & (self.target < self.V))
        assert bool((o["loss"][~keep] == 0).all()) and bool((o["lse"][~keep] == 0).all())
        norm = 1.0
        if self.mean:
            norm = abs(float(m["w"].sum())) or 1.0
        assert abs(float(o["total"][0]) - float(ref["total"])) <= float(row.sum()) / norm + 2.0 ** -23 * abs(float(ref["total"]))
        if not grads:
            return ref
        top = float((m["gw"] * torch.clamp(m["zf"], min=1)).max()) if m["keep"].numel() else 0.0
        tiny = top * 2.0 ** -13 * 2.0 ** -25  # dl rounded among f16's subnormals
        e = u * m["d"] + (2 * logit + 2.0 ** -19) * (m["p"] + m["d"]) + tiny
        for k in which:
            if k == "dH":
                bound = torch.zeros_like(ref["dH"])
                bound[m["keep"]] = c * (e @ m["Wd"].abs() + acc(self.V) * 2 * (m["d"] @ m["Wd"].abs()))
            else:
                bound = c * (e.T @ m["Hd"].abs() + acc(self.T) * 2 * (m["d"].T @ m["Hd"].abs()))
            bound += u * ref[k].abs() + 2.0 ** -25
            off = (o[k].double() - ref[k]).abs()
            assert bool((off <= bound).all()), (k, float((off / bound).max()))
            # roundings are independent: in the 2-norm they stay well below their bound
            size = float(ref[k].norm())
            if self.ab == "bf16" and size > 0 and ref[k].numel() > 2000:
                assert float(off.norm()) <= 1.0 * u * size, (k, float(off.norm()) / size)
        return ref

    clean = False


SIZES = [(1, 1, 1), (1, 300, 64), (2, 257, 8), (3, 1000, 17), (31, 129, 100), (64, 2048, 512), (127, 640, 130), (128, 4096, 256),
         (129, 777, 72), (200, 5000, 320), (256, 256, 256), (257, 1025, 65), (600, 3333, 200), (1000, 2000, 1111)]


@pytest.mark.gpu
@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_step_sizes(T, V, D, ab):
    c = Case(T, V, D, ab, seed=T + V + D, g=64.0 if ab == "f16" else 1.0)
    c.check(c.step())


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,D", SIZES)
def test_loss_sizes_and_same_bits_as_step(T, V, D):
    c = Case(T, V, D, seed=T * 3 + V)
    o = c.loss()
    c.check(o, grads=False)
    s = c.step()
    for k in ("loss", "lse", "total"):
        assert torch.equal(o[k], s[k])


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    dict(ignored=0.5), dict(ignored=0.97), dict(weights="positive", mean=False), dict(weights="mixed", z=1e-3),
    dict(weights="zero"), dict(c=0.25, z=0.01), dict(c=-0.5), dict(c=1.7, mean=False, g=-3.0), dict(z=0.5, scale=6.0),
    dict(index="i32", ignored=0.2), dict(pad=(1, 2, 3, 4)), dict(scale=12.0), dict(scale=0.0), dict(max_ctas=5), dict(max_ctas=1),
    dict(z=20.0, ab="f16")], ids=str)
@pytest.mark.parametrize("T,V,D", [(77, 1100, 96), (300, 1300, 200)])
def test_step_options(T, V, D, kw):
    c = Case(T, V, D, seed=5, **kw)
    c.check(c.step())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 300])
def test_pieces_of_the_vocabulary(T):
    # 256 columns at a time: full pieces, and one that ends inside a tile and a k-block
    c = Case(T, 1999, 120, seed=1, buffer_bytes=1, ignored=0.1)
    c.check(c.step())


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(), dict(ignored=0.3, buffer_bytes=1777 * 2 * 2048), dict(weights="positive", z=1e-3)], ids=str)
def test_step_of_many_fp16_rows(kw):
    # four products, three of them after one another for each piece
    c = Case(1777, 6001, 304, "f16", seed=3, g=256.0, **kw)
    c.check(c.step())


@pytest.mark.gpu
@pytest.mark.parametrize("ab", ["bf16", "f16"])
@pytest.mark.parametrize("D", [1280, 1536, 4096])
def test_sums_of_a_long_width_are_taken_in_runs(D, ab):
    """The tensor unit's fp32 sums are cut off, which lowers lse by 4.8e-10 of itself for every column in a run (bf16;
    fp16 a quarter more).  Runs hold it to what 1024 columns of bf16 lose; beside that mean there are only roundings of
    either sign."""
    T, V = 300, 8000
    c = Case(T, V, D, ab, seed=D, scale=2.5)
    near = torch.arange(0, T, 2, device=c.H.device)
    c.H[near] += c.W[c.target[near]]
    o = c.loss()
    ref = c.check(o, grads=False)
    assert abs(float((o["lse"].double() / ref["lse"] - 1).mean())) <= 4.8e-10 * 1024 + 2.0 ** -24


# up to 128 rows: bands of columns whose last tile ends past the vocabulary, or which a piece's end cuts
BANDS = [(2, 32000, {}), (64, 32000, {}), (128, 32000, {}), (64, 32768, {}), (2, 51200, {}), (128, 51200, {}), (64, 131072, {}),
         (2, 262144, {}), (64, 10000, dict(buffer_bytes=1)), (64, 10240, dict(buffer_bytes=1)), (128, 1024, dict(max_ctas=6)),
         (64, 10000, dict(max_ctas=19, buffer_bytes=1)), (40, 32000, dict(max_ctas=19, ignored=0.2))]


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,kw", BANDS, ids=str)
def test_bands_over_a_vocabulary(T, V, kw):
    c = Case(T, V, 24, seed=T + V, **kw)
    first = c.step()
    c.check(first)
    again = c.step()
    for k in first:
        assert torch.equal(first[k], again[k]), k


@pytest.mark.gpu
@pytest.mark.parametrize("c,buffer_bytes", [(1.0, 0), (-0.5, 0), (1.0, 1)])
@pytest.mark.parametrize("T", [40, 300])
def test_words_of_no_probability(T, c, buffer_bytes):
    """Words whose logit is 64 below their neighbours' have p = 2e-28: no gradient of theirs is seen beside 2^-38 of
    a row's.  All logits are exact in fp32; a kept distance moves p by at most 2^-12 of itself."""
    V, D = 512, 8
    gen = torch.Generator().manual_seed(T)
    s = Case(T, V, D, c=c, mean=False, buffer_bytes=buffer_bytes)
    s.H.copy_(torch.randint(-8, 9, (T, D), generator=gen).to(s.H))
    s.H[:, 0] = 64.0
    s.W.zero_()
    s.W[[5, 70, 130, 300, 511], 0] = 1 / c
    s.target.copy_(torch.randint(256, 300, (T,), generator=gen))
    o = s.step()
    torch.cuda.synchronize()
    ref, m = reference(s.H, s.W, s.target, None, c, 0.0, False, 1.0)
    e = U["bf16"] * m["d"] + 2.0 ** -12 * m["p"] + 2.0 ** -38
    for k, off in (("dH", e @ m["Wd"].abs()), ("dW", e.T @ m["Hd"].abs())):
        bound = abs(c) * off * (1 + 2.0 ** -10) + U["bf16"] * ref[k].abs()
        assert bool(((o[k].double() - ref[k]).abs() <= bound).all()), k


@pytest.mark.gpu
@pytest.mark.parametrize("ab,c,pieces", [("bf16", 1.0, 1), ("bf16", -0.5, 1), ("bf16", 1.0, 2), ("bf16", -0.25, 2), ("f16", 1.0, 1)])
@pytest.mark.parametrize("T", [40, 300])
def test_logits_of_thousands(T, ab, c, pieces):
    """Largest logits of 2000 to 16000 that are not the target's.  They and the differences between them are exact in
    fp32; in log2 units they are below 2^15, so that rounding lse moves p by at most 2^-10 of itself, and a kept
    distance by 2^-12: 2^-9 of p in all, beside the roundings of dl and of the results."""
    V, D = 512, 8
    gen = torch.Generator().manual_seed(T)
    s = Case(T, V, D, ab, c=c, mean=False, buffer_bytes=1 if pieces == 2 else 0)
    s.H.zero_()
    s.W.zero_()
    s.H[:, 0] = (torch.randint(128, 256, (T,), generator=gen) * 2.0 ** torch.randint(4, 7, (T,), generator=gen)).to(s.H)
    s.H[:, 1] = 1.0
    near = torch.tensor([5, 6, 70, 130, 250, 300, 511])
    s.W[near, 0] = 1 / c
    s.W[near, 1] = torch.tensor([0.0, -0.25, -1.0, -0.5, 0.0, -0.75, -2.0]).to(s.W) / c
    s.W[:, 2:] = (torch.randint(-8, 9, (V, D - 2), generator=gen) / 8).to(s.W)  # seen by dH alone
    s.target.copy_(torch.randint(7, 60, (T,), generator=gen))
    o = s.step()
    torch.cuda.synchronize()
    assert B.gemm_epi_last_error() == B.GE_OK
    ref, m = reference(s.H, s.W, s.target, None, c, 0.0, False, 1.0)
    assert bool(((o["lse"].double() - ref["lse"]).abs() <= 2.0 ** -20 * ref["lse"]).all())
    e = U[ab] * m["d"] + 2.0 ** -9 * m["p"] + 2.0 ** -38
    for k, off in (("dH", e @ m["Wd"].abs()), ("dW", e.T @ m["Hd"].abs())):
        bound = abs(c) * off * (1 + 2.0 ** -10) + U[ab] * ref[k].abs() + 2.0 ** -24
        past = torch.isinf(o[k]) & (ref[k].abs() > torch.finfo(TYPE[ab]).max)  # no number of the type
        assert bool((past | ((o[k].double() - ref[k]).abs() <= bound)).all()), k


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 50, 300])
def test_all_rows_ignored(T):
    c = Case(T, 500, 64, ignored=2.0)
    o = c.step()
    c.check(o)
    assert float(o["total"][0]) == 0 and not bool(o["dH"].any()) and not bool(o["dW"].any())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [60, 400])
def test_ignored_rows_may_hold_anything(T):
    c = Case(T, 700, 80, seed=3, ignored=0.4)
    gone = c.target < 0
    c.H[gone] = float("nan")
    c.H[gone.nonzero()[::2, 0]] = float("inf")
    c.clean = True
    c.check(c.step())


@pytest.mark.gpu
def test_targets_outside_the_vocabulary_are_ignored():
    c = Case(50, 300, 64, seed=4)
    c.target[::5] = torch.tensor([300, -1, 1 << 40, -(1 << 40), 301, 299, 0, -100, 4294967295, 2147483648], device=c.H.device)
    c.check(c.step())


@pytest.mark.gpu
def test_nan_and_infinity_stay_in_their_rows():
    c = Case(200, 900, 64, seed=6, mean=False)
    c.H[7, 3] = float("nan")
    c.H[150, 0] = float("inf")  # logits of both signs of infinity
    o = c.step()
    torch.cuda.synchronize()
    bad = torch.zeros(200, dtype=torch.bool, device=c.H.device)
    bad[[7, 150]] = True
    assert bool(torch.isnan(o["loss"][bad]).all()) and bool(torch.isfinite(o["loss"][~bad]).all())
    assert bool(torch.isnan(o["dH"][bad]).any(1).all()) and bool(torch.isfinite(o["dH"][~bad]).all())
    assert bool(torch.isnan(o["total"]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [100, 300])
def test_one_gradient_alone(T):
    c = Case(T, 800, 96, seed=8)
    both = c.step()
    h = c.step(dW=False)
    c.check(h, which=("dH",))
    assert torch.equal(h["dH"], both["dH"]) and bool((h["dW"] == 77).all())
    w = c.step(dH=False)
    c.check(w, which=("dW",))
    assert torch.equal(w["dW"], both["dW"]) and bool((w["dH"] == 77).all())


@pytest.mark.gpu
def test_repeats_bit_for_bit_whatever_the_workspace_held():
    c = Case(333, 2500, 128, seed=9, ignored=0.3, buffer_bytes=333 * 2 * 1024)
    ws = c.workspace(True)
    first = c.step(ws=ws)
    c.H, keep = c.H.clone().mul_(0.5), c.H
    c.step(ws=ws)
    c.H = keep
    again = c.step(ws=ws)
    for k in first:
        assert torch.equal(first[k], again[k]), k


@pytest.mark.gpu
def test_another_stream_and_a_graph():
    c = Case(150, 1200, 64, seed=10)
    want = c.step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = c.step(stream=side)
    side.synchronize()
    for k in want:
        assert torch.equal(want[k], got[k])
    o, ws = c.outputs(), c.workspace(True)
    call = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call = B.prepare_xent_step(c.plan, c.H, c.W, c.target, None, 1.0, o["loss"], o["lse"], o["total"], o["dH"], o["dW"], ws)
        assert call() == B.GE_OK
    c.H.mul_(0.25)
    graph.replay()
    torch.cuda.synchronize()
    c.check(o)


@pytest.mark.gpu
def test_long_rows_of_offsets_past_32_bits():
    # the last rows of a W of more than 2^31 elements decide this loss
    V, D = 70001, 32768
    dev = torch.device("cuda", 0)
    W = torch.zeros(V, D, dtype=torch.bfloat16, device=dev)
    W[-3:, -40:] = 1.0
    H = torch.zeros(4, D, dtype=torch.bfloat16, device=dev)
    H[:, -40:] = 0.5
    t = torch.tensor([V - 1, V - 2, 0, V - 4], device=dev)
    plan = B.gemm_epi_xent_plan_create(4, V, D, B.make_xent_desc("bf16"))
    dW, dH = torch.full_like(W, 5.0), torch.empty_like(H)
    loss, lse, total = torch.empty(4, device=dev), torch.empty(4, device=dev), torch.empty(1, device=dev)
    ws = torch.empty(B.gemm_epi_xent_workspace_bytes(plan, True), dtype=torch.uint8, device=dev)
    B.gemm_epi_xent_step(plan, H, W, t, None, 1.0, loss, lse, total, dH, dW, ws)
    torch.cuda.synchronize()
    n = np.log((V - 3) + 3 * np.exp(20.0))
    assert np.allclose(lse.cpu().numpy(), n, rtol=2.0 ** -19)
    assert np.allclose(loss.cpu().numpy(), [n - 20, n - 20, n, n], atol=2.0 ** -14)
    p = np.exp(20.0 - n)
    want = np.array([p, p - 0.25, p - 0.25]) * 0.5  # each column's mean of p - [target], times H
    # the rows' dl, each off by 2^-8, add up to five times what is left of them
    assert np.allclose(dW[-3:, -1].float().cpu().numpy(), want, rtol=2.0 ** -5)
    assert float(dW[-3:, :-40].abs().max()) == 0
    B.gemm_epi_xent_plan_destroy(plan)


@pytest.mark.gpu
def test_a_vocabulary_of_more_column_blocks_than_a_grid_has_rows():
    # 512 columns each, and 65535: a step that keeps the logits of 33.6 million words
    T, V, D = 2, 33_600_000, 8
    dev = torch.device("cuda", 0)
    gen = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randn(V, D, generator=gen, device=dev, dtype=torch.bfloat16)
    H = torch.randn(T, D, generator=gen, device=dev, dtype=torch.bfloat16)
    t = torch.tensor([V - 1, 77], device=dev)
    plan = B.gemm_epi_xent_plan_create(T, V, D, B.make_xent_desc("bf16", reduction="sum"))
    ws = torch.full((B.gemm_epi_xent_workspace_bytes(plan, True),), 0xFF, dtype=torch.uint8, device=dev)
    loss, lse, total, dW, dH = torch.empty(T, device=dev), torch.empty(T, device=dev), None, torch.full_like(W, 7.0), torch.empty_like(H)
    assert B.gemm_epi_xent_step(plan, H, W, t, None, 1.0, loss, lse, total, dH, dW, ws, check=False) == B.GE_OK
    torch.cuda.synchronize()
    assert B.gemm_epi_last_error() == B.GE_OK
    l = H.double() @ W.double().T
    want = torch.logsumexp(l, 1)
    assert bool(((lse.double() - want).abs() <= 2.0 ** -18 * want).all())
    d = torch.exp(l - want[:, None])
    d[torch.arange(T), t] -= 1
    mag = H.double().abs()
    for first in (0, V // 2, V - 4096):  # dl, its products with H and their sum are rounded to bf16, p is off by 2^-12
        at = slice(first, first + 4096)
        bound = (2 * U["bf16"] + 2.0 ** -10) * (d[:, at].abs().T @ mag) + 2.0 ** -60
        assert bool(((dW[at].double() - d[:, at].T @ H.double()).abs() <= bound).all()), first
    bound = (U["bf16"] + 2.0 ** -10 + 2 * acc(V)) * (d.abs() @ W.double().abs()) + U["bf16"] * (d @ W.double()).abs()
    assert bool(((dH.double() - d @ W.double()).abs() <= bound).all())
    B.gemm_epi_xent_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [20, 300])
def test_a_load_that_never_comes_is_reported(T):
    """The first k-block of every product is left out: its wait runs out after 20 ms and the run ends by itself."""
    c = Case(T, 600, 128, seed=12)
    plan, desc = c.plan, B.make_xent_desc("bf16", timeout_ms=20, debug_flags=B.GE_DEBUG_SKIP_FIRST_LOAD)
    c.plan = B.gemm_epi_xent_plan_create(T, 600, 128, desc)
    c.step()
    torch.cuda.synchronize()
    assert B.gemm_epi_last_error() == B.GE_ERR_TIMEOUT
    B.gemm_epi_xent_plan_destroy(c.plan)
    c.plan = plan
    c.check(c.step())


def test_gradient_formula_against_differences():
    gen = torch.Generator().manual_seed(2)
    T, V, D = 5, 11, 7
    H, W = torch.randn(T, D, generator=gen, dtype=torch.float64), torch.randn(V, D, generator=gen, dtype=torch.float64)
    t = torch.tensor([3, -100, 0, 10, 7])
    w = torch.randn(T, generator=gen, dtype=torch.float64)

    def total(H, W):
        return float(reference(H, W, t, w, 0.7, 0.05, True, 1.0)[0]["total"])

    ref, _ = reference(H, W, t, w, 0.7, 0.05, True, 1.0)
    h = 1e-5
    for X, k in ((H, "dH"), (W, "dW")):
        for i in range(X.shape[0]):
            for j in range(X.shape[1]):
                up, dn = X.clone(), X.clone()
                up[i, j] += h
                dn[i, j] -= h
                d = (total(up, W) - total(dn, W)) / (2 * h) if X is H else (total(H, up) - total(H, dn)) / (2 * h)
                assert abs(d - float(ref[k][i, j])) < 1e-8


def _create(T=4, V=8, D=8, **kw):
    return B.gemm_epi_xent_plan_create(T, V, D, B.make_xent_desc(**{"ab": "bf16", **kw}))


@pytest.mark.parametrize("kw,status", [
    (dict(ab="f32"), "UNSUPPORTED"), (dict(index=2), "UNSUPPORTED"), (dict(T=0), "SHAPE"), (dict(V=0), "SHAPE"), (dict(D=-1), "SHAPE"),
    (dict(T=1 << 31), "SHAPE"), (dict(ldh=7), "SHAPE"), (dict(D=9), "MISALIGNED"), (dict(ldw=12), "MISALIGNED"),
    (dict(reduction=2), "INVALID"), (dict(timeout_ms=-1), "INVALID"), (dict(logit_scale=float("nan")), "INVALID"),
    (dict(z_loss=float("inf")), "INVALID"), (dict(buffer_bytes=-1), "INVALID"), (dict(max_ctas=-2), "INVALID"),
    (dict(debug_flags=2), "INVALID")], ids=str)
def test_plan_refusals(kw, status):
    with pytest.raises(B.GemmEpiError) as e:
        _create(**kw)
    assert e.value.status == getattr(B, "GE_ERR_" + status)


def test_null_plans():
    assert B.lib.gemm_epi_xent_plan_create(None, 1, 1, 8, None) == B.GE_ERR_INVALID
    assert B.gemm_epi_xent_workspace_bytes(None, True) == 0
    assert B.lib.gemm_epi_xent_loss(None, *[None] * 8, 0, None) == B.GE_ERR_INVALID
    B.gemm_epi_xent_plan_destroy(None)


@pytest.mark.gpu
def test_run_refusals():
    c = Case(8, 64, 64)
    o, ws = c.outputs(), c.workspace(True)

    def step(**kw):
        a = dict(H=c.H, W=c.W, target=c.target, weight=None, grad_scale=1.0, loss=o["loss"], lse=o["lse"], total=o["total"],
                 dH=o["dH"], dW=o["dW"], workspace=ws, check=False)
        a.update(kw)
        return B.gemm_epi_xent_step(c.plan, **a)

    assert step(H=None) == step(W=None) == step(target=None) == step(dH=None, dW=None) == B.GE_ERR_MISSING_ARG
    for k in ("H", "W", "target", "loss", "dH", "dW"):
        p = {"H": c.H, "W": c.W, "target": c.target}.get(k, o.get(k)).data_ptr()
        assert step(**{k: p + 8}) == B.GE_ERR_MISALIGNED, k
    assert step(workspace=None, workspace_bytes=1 << 30) == B.GE_ERR_WORKSPACE
    assert step(workspace_bytes=ws.numel() - 1) == B.GE_ERR_WORKSPACE
    assert step(grad_scale=float("nan")) == B.GE_ERR_INVALID
    assert step(loss=None, lse=None, total=None) == B.GE_OK
    torch.cuda.synchronize()
