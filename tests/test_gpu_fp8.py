"""Block-scaled 8-bit products against 64 bits.

Bounds, derived before any run.  Products of 8-bit floats are exact.  A block's 128 products are summed in fp32 by
additions that may cut off: at most 2^-23 of the magnitudes for each, 2^-16 in all.  The scales' product, the scaled sum
and its addition round once each (2^-24) for each block, slices once more: (blocks + 4) 2^-23 of the magnitudes.  The
result is rounded once (u).
"""
import pytest
import torch

from dense_gemm_elementwise_gb300 import build as gbuild

gbuild.build()
from dense_gemm_elementwise_gb300 import binding as B  # noqa: E402

TYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
        "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -130, "f32": 2.0 ** -130}
SENT = 77.0


def blocks(n):
    return -(-n // 128)


def up(n, m):
    return -(-n // m) * m


class Case:
    def __init__(self, M, N, K, a="e4m3", b="e4m3", d="bf16", block="square", add=False, pad=(0, 0, 0), more_scales=0,
                 max_ctas=0, seed=0, small=1.0, **kw):
        g = torch.Generator(device="cuda").manual_seed(seed + M * 7 + N * 3 + K)
        dev = torch.device("cuda", 0)
        self.M, self.N, self.K, self.d, self.square = M, N, K, d, block == "square"
        lda, ldb = up(K, 16) + 16 * pad[0], up(K, 16) + 16 * pad[1]

        def eight(rows, ld, kind):
            # between the rows lies NaN
            v = torch.full((rows, ld), 0x7F, dtype=torch.uint8, device=dev)
            x = (torch.randn(rows, K, generator=g, device=dev) * (LARGEST[kind] / 4)).clamp(-LARGEST[kind], LARGEST[kind])
            v[:, :K] = x.to(TYPE[kind]).view(torch.uint8)
            return v.view(TYPE[kind])[:, :K]

        def scales(*shape):
            s = torch.full((shape[0], shape[1] + more_scales), float("nan"), device=dev)
            s[:, :shape[1]] = (torch.randn(*shape, generator=g, device=dev) - 9).exp() * small
            return s[:, :shape[1]]

        self.A, self.B = eight(M, lda, a), eight(N, ldb, b)
        self.sa = scales(blocks(K), M)
        self.sb = scales(blocks(K), blocks(N) if self.square else N)
        self.ldd = N + pad[2]
        self.C = None
        if add:
            self.C = torch.full((M, self.ldd), float("nan"), dtype=TYPE[d], device=dev)[:, :N]
            self.C.copy_(torch.randn(M, N, generator=g, device=dev) * 10 * K ** 0.5)
        self.buf = torch.full((M + 2, self.ldd), SENT, dtype=TYPE[d], device=dev)
        self.desc = B.make_fp8_desc(a, b, d, b_block=block, lda=lda, ldb=ldb, ldd=self.ldd, lds_a=M + more_scales,
                                    lds_b=self.sb.shape[1] + more_scales, max_ctas=max_ctas, **kw)
        self.plan = B.gemm_epi_fp8_plan_create(M, N, K, self.desc)
        n = B.gemm_epi_fp8_workspace_bytes(self.plan)
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev) if n else None

    @property
    def D(self):
        return self.buf[1:-1, :self.N]

    def run(self, D=None, C=None, stream=None):
        out = self.buf[1:] if D is None else D
        if self.ldd * out.element_size() % 16:  # a row's start that is not aligned: from the buffer's own
            out = self.buf if D is None else D
        self.at = 0 if out is self.buf else 1
        B.gemm_epi_fp8_run(self.plan, self.A, self.sa, self.B, self.sb, self.C if C is None else C, out, self.ws, stream=stream)
        return self

    def want(self):
        A = self.A.double() * self.sa.double().t().repeat_interleave(128, 1)[:, :self.K]
        sb = self.sb.double()
        if self.square:
            sb = sb.repeat_interleave(128, 1)[:, :self.N]
        Bm = self.B.double() * sb.t().repeat_interleave(128, 1)[:, :self.K]
        y, mag = A @ Bm.t(), A.abs() @ Bm.abs().t()
        if self.C is not None:
            y, mag = y + self.C.double(), mag + self.C.double().abs()
        return y, mag

    def check(self, got=None, want=None):
        torch.cuda.synchronize()
        assert B.gemm_epi_last_error() == B.GE_OK
        if got is None:
            got = self.buf[self.at:self.at + self.M, :self.N]
            rest = torch.ones_like(self.buf, dtype=torch.bool)
            rest[self.at:self.at + self.M, :self.N] = False
            assert bool((self.buf[rest] == SENT).all()), "write outside the output"
        y, mag = want or self.want()
        lim = mag * (2.0 ** -16 + (blocks(self.K) + 4) * 2.0 ** -23) + y.abs() * U[self.d] + TINY[self.d]
        off = (got.double() - y).abs()
        worst = (off / lim).max().item()
        assert worst <= 1.0 and not bool(got.isnan().any()), (worst, (off > lim).nonzero()[:4].tolist())
        B.gemm_epi_fp8_plan_destroy(self.plan)


SIZES = [(1, 1, 1), (1, 64, 128), (2, 8, 16), (5, 130, 200), (8, 1000, 129), (16, 16, 4096), (17, 300, 385), (33, 129, 1000), (64, 512, 512),
         (65, 200, 130), (127, 128, 128), (128, 128, 256), (129, 300, 1000), (200, 4000, 640), (256, 256, 128), (257, 513, 385),
         (512, 2560, 300), (700, 1000, 2000), (1000, 5000, 130)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("block", ["square", "row"])
def test_sizes(M, N, K, block):
    Case(M, N, K, block=block).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("a", ["e4m3", "e5m2"])
@pytest.mark.parametrize("b", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M,N", [(3, 200), (100, 136), (300, 5000)])
def test_types_of_operands(a, b, M, N):
    # (e5m2's largest products times their scales stay within fp16)
    Case(M, N, 300, a, b, "f16", small=2.0 ** -7 if a == b == "e4m3" else 2.0 ** -20).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("d", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K,pad", [(1, 700, 500, (1, 2, 8)), (40, 700, 500, (1, 0, 3)), (300, 704, 260, (0, 1, 0)), (300, 701, 260, (0, 1, 0)),
                                       (600, 5001, 260, (2, 1, 1)), (600, 5008, 260, (0, 0, 0))])
@pytest.mark.parametrize("block", ["square", "row"])
def test_outputs_sums_and_pitches(d, M, N, K, pad, block):
    Case(M, N, K, d=d, block=block, add=True, pad=pad, more_scales=3, small=2.0 ** -7).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(1, 100), (1, 3000), (20, 2500), (130, 300), (128, 1290)])
@pytest.mark.parametrize("K", [128, 256, 1152, 1408, 2000, 5000])
def test_sums_split_among_the_ctas_of_a_cluster(M, N, K):
    """Numbers of k-blocks that the slices do and do not divide."""
    Case(M, N, K, d="f32", add=True, block="row").run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(5, 300, 1000), (300, 300, 700), (600, 5000, 400)])
def test_sum_in_place(M, N, K):
    c = Case(M, N, K, d="f32", add=True)
    want = c.want()
    B.gemm_epi_fp8_run(c.plan, c.A, c.sa, c.B, c.sb, c.C, c.C, c.ws)
    c.check(c.C, want)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(600, 4992, 400), (590, 5000, 130), (1300, 2100, 2100), (130, 700, 150)])
@pytest.mark.parametrize("d", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block", ["square", "row"])
def test_large_sums_added(M, N, K, d, block):
    Case(M, N, K, d=d, block=block, add=True, pad=(0, 0, 8), seed=9).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 2, 3, 7, 8, 9, 13, 16])
@pytest.mark.parametrize("N,K,ctas", [(6, 2, 0), (40, 100, 0), (129, 128, 0), (300, 2100, 2), (900, 1160, 3), (5500, 1024, 0), (9800, 390, 0), (80000, 130, 0)])
@pytest.mark.parametrize("block", ["square", "row"])
def test_few_rows(M, N, K, ctas, block):
    Case(M, N, K, block=block, max_ctas=ctas, more_scales=1, seed=5).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 20])
@pytest.mark.parametrize("block", ["square", "row"])
def test_many_tiles_for_a_cta(ctas, block):
    """Scales and accumulators change hands from tile to tile with odd and even numbers of k-blocks."""
    Case(600, 900, 640, block=block, max_ctas=ctas).run().check()
    Case(300, 700, 130, block=block, max_ctas=ctas).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(3, 500, 900), (140, 300, 900), (600, 4900, 300)])
def test_nan_stays_in_its_row_and_column(M, N, K):
    c = Case(M, N, K, d="f32")
    c.A.view(torch.uint8)[1, 5] = 0x7F
    c.B.view(torch.uint8)[7, 130] = 0xFF
    c.sb[0, 1] = float("inf")
    c.run()
    torch.cuda.synchronize()
    got = c.buf[c.at:c.at + M, :N]
    fine = torch.ones(M, N, dtype=torch.bool, device=got.device)
    fine[1] = fine[:, 7] = False
    fine[:, 128:256] = False
    assert bool(got[1].isnan().all()) and bool(got[:, 7].isnan().all())
    assert bool(got[fine].isfinite().all()) and not bool(got[:, 128:256].isfinite().any())


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (30, 500, 2000), (257, 513, 385), (600, 5000, 400)])
def test_another_stream_a_graph_and_the_same_bits(M, N, K):
    c = Case(M, N, K, d="f32")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    torch.cuda.synchronize()
    first = c.buf.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(stream=torch.cuda.current_stream())
    for fill in (0xFF, 0x55):
        c.buf.fill_(SENT)
        if c.ws is not None:
            c.ws.fill_(fill)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, c.buf)
    c.sa *= 2.0  # another input, in place
    graph.replay()
    c.check()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    M, N, K = 40000, 60000, 16
    dev = torch.device("cuda", 0)
    c = Case(256, 512, K, d="f16", small=2.0 ** -7)
    A, Bm = torch.zeros(M, K, dtype=torch.uint8, device=dev), torch.zeros(N, K, dtype=torch.uint8, device=dev)
    A[-256:], Bm[-512:] = c.A.view(torch.uint8), c.B.view(torch.uint8)
    sa, sb = torch.ones(1, M, device=dev), torch.ones(1, N, device=dev)
    sa[:, -256:] = c.sa
    sb[:, -512:] = c.sb.repeat_interleave(128, 1)
    plan = B.gemm_epi_fp8_plan_create(M, N, K, B.make_fp8_desc("e4m3", "e4m3", "f16", b_block="row"))
    D = torch.empty(M, N, dtype=torch.float16, device=dev)
    n = B.gemm_epi_fp8_workspace_bytes(plan)
    B.gemm_epi_fp8_run(plan, A, sa, Bm, sb, None, D, torch.empty(n, dtype=torch.uint8, device=dev) if n else None)
    torch.cuda.synchronize()
    B.gemm_epi_fp8_plan_destroy(plan)
    assert not bool(D[:-256].any()) and not bool(D[:, :-512].any())
    c.check(D[-256:, -512:])


@pytest.mark.gpu
@pytest.mark.parametrize("M,N", [(100, 200), (600, 5000)])
def test_a_load_that_never_comes_is_reported(M, N):
    c = Case(M, N, 1000, timeout_ms=50, debug_flags=B.GE_DEBUG_SKIP_FIRST_LOAD)
    c.run()
    torch.cuda.synchronize()
    assert B.gemm_epi_last_error() == B.GE_ERR_TIMEOUT
    B.gemm_epi_fp8_plan_destroy(c.plan)
    Case(M, N, 1000).run().check()


def bad(M=100, N=100, K=64, a="e4m3", b="e4m3", d="bf16", **kw):
    reserved = kw.pop("reserved", 0)
    r = B.make_fp8_desc(a, b, d, **kw)
    r.reserved = reserved
    with pytest.raises(B.GemmEpiError) as e:
        B.gemm_epi_fp8_plan_create(M, N, K, r)
    return e.value.status


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), "GE_ERR_SHAPE"), (dict(N=-1), "GE_ERR_SHAPE"), (dict(K=1 << 31), "GE_ERR_SHAPE"),
    (dict(a="bf16"), "GE_ERR_UNSUPPORTED"), (dict(b=7), "GE_ERR_UNSUPPORTED"), (dict(d="e4m3"), "GE_ERR_UNSUPPORTED"),
    (dict(b_block=2), "GE_ERR_INVALID"), (dict(timeout_ms=-1), "GE_ERR_INVALID"), (dict(max_ctas=-1), "GE_ERR_INVALID"),
    (dict(debug_flags=2), "GE_ERR_INVALID"), (dict(reserved=1), "GE_ERR_INVALID"), (dict(lda=48), "GE_ERR_SHAPE"),
    (dict(K=65), "GE_ERR_MISALIGNED"), (dict(lda=72), "GE_ERR_MISALIGNED"), (dict(ldb=72), "GE_ERR_MISALIGNED"),
    (dict(ldd=99), "GE_ERR_SHAPE"), (dict(lds_a=99), "GE_ERR_SHAPE"), (dict(lds_b=99, b_block="row"), "GE_ERR_SHAPE")])
def test_plan_refusals(kw, status):
    assert bad(**kw) == getattr(B, status)


def test_null_plans():
    assert B.lib.gemm_epi_fp8_plan_create(None, 1, 1, 1, None) == B.GE_ERR_INVALID
    assert B.lib.gemm_epi_fp8_run(*[None] * 8, 0, None) == B.GE_ERR_INVALID
    assert B.gemm_epi_fp8_workspace_bytes(None) == 0
    B.gemm_epi_fp8_plan_destroy(None)


@pytest.mark.gpu
def test_run_refusals():
    c = Case(300, 300, 4096)
    run = lambda A=c.A, sa=c.sa, Bm=c.B, sb=c.sb, C=None, D=c.buf, ws=None: B.gemm_epi_fp8_run(  # noqa: E731
        c.plan, A, sa, Bm, sb, C, D, ws, 0, check=False)
    for name in ("A", "sa", "Bm", "sb", "D"):
        assert run(**{name: 0}) == B.GE_ERR_MISSING_ARG
    for name, t in (("A", c.A), ("Bm", c.B), ("C", c.buf), ("D", c.buf)):
        assert run(**{name: t.data_ptr() + 8}) == B.GE_ERR_MISALIGNED
    assert run(sa=c.sa.data_ptr() + 2) == B.GE_ERR_MISALIGNED
    assert run(ws=c.buf.data_ptr() + 8) == B.GE_ERR_MISALIGNED


@pytest.mark.gpu
def test_a_linear_layer_forward_and_backward():
    """What the quantiser makes, through the layer's three products, against 64 bits of the same 8-bit values; and
    against the unquantised layer: two roundings of 2^-4 at most for each product, independent, so that in the
    2-norm a result is off by less than 2 * 2^-4."""
    T, K, N = 390, 520, 264
    dev = torch.device("cuda", 0)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, W, dy = (torch.randn(*s, generator=g, device=dev).to(torch.bfloat16) for s in ((T, K), (N, K), (T, N)))

    def quantised(v, block, rows, cols):
        n, k = v.shape
        plan = B.gemm_epi_quant_plan_create(n, k, B.make_quant_desc("bf16", "e4m3", block=block, ldq=up(k, 16), ldqt=up(n, 16)))
        side = (lambda m: blocks(m)) if block == "square" else (lambda m: m)
        q, s = torch.empty(n, up(k, 16), dtype=torch.uint8, device=dev), torch.empty(blocks(k), side(n), device=dev)
        qt, st = torch.empty(k, up(n, 16), dtype=torch.uint8, device=dev), torch.empty(blocks(n), side(k), device=dev)
        B.gemm_epi_quant_run(plan, v, q if rows else None, s if rows else None, qt if cols else None, st if cols else None)
        torch.cuda.synchronize()
        B.gemm_epi_quant_plan_destroy(plan)
        return (q, s), (qt, st)

    def product(a, b, M, N, K, d, block, C=None):
        plan = B.gemm_epi_fp8_plan_create(M, N, K, B.make_fp8_desc("e4m3", "e4m3", d, b_block=block, lda=up(K, 16), ldb=up(K, 16)))
        n = B.gemm_epi_fp8_workspace_bytes(plan)
        D = torch.empty(M, N, dtype=TYPE[d], device=dev)
        B.gemm_epi_fp8_run(plan, a[0], a[1], b[0], b[1], C, D, torch.empty(n, dtype=torch.uint8, device=dev) if n else None)
        torch.cuda.synchronize()
        B.gemm_epi_fp8_plan_destroy(plan)
        return D

    def value(a, n, k, square=False):
        s = a[1].double().t().repeat_interleave(128, 1)[:, :k]
        if square:
            s = s.repeat_interleave(128, 0)[:n]
        return a[0][:, :k].contiguous().view(torch.float8_e4m3fn).double() * s

    qx, qxt = quantised(x, "row", True, True)
    qw, qwt = quantised(W, "square", True, True)
    qd, qdt = quantised(dy, "row", True, True)
    dW0 = torch.randn(N, K, generator=g, device=dev)
    y = product(qx, qw, T, N, K, "bf16", "square")
    dx = product(qd, qwt, T, K, N, "bf16", "square")
    dW = product(qdt, qxt, N, K, T, "f32", "row", C=dW0)
    assert B.gemm_epi_last_error() == B.GE_OK
    for got, a, b, k, d, plain in (
            (y, value(qx, T, K), value(qw, N, K, True), K, "bf16", x.double() @ W.double().t()),
            (dx, value(qd, T, N), value(qwt, K, N, True), N, "bf16", dy.double() @ W.double()),
            (dW - dW0, value(qdt, N, T), value(qxt, K, T), T, "f32", dy.double().t() @ x.double())):
        ref, mag = a @ b.t(), a.abs() @ b.abs().t()
        if d == "f32":
            mag = mag + 2 * dW0.double().abs()
        lim = mag * (2.0 ** -16 + (blocks(k) + 4) * 2.0 ** -23) + ref.abs() * U[d]
        assert bool(((got.double() - ref).abs() <= lim).all())
        assert float((got.double() - plain).norm() / plain.norm()) <= 2.0 ** -3


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 300, 385), (7, 1000, 260), (16, 300, 385), (17, 300, 385), (100, 136, 128), (130, 700, 1500), (600, 5000, 260)])
@pytest.mark.parametrize("block", ["square", "row"])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("ea,eb,least", [(-60, -62, False), (-30, -90, False), (-90, -30, False), (-100, 87, False), (120, -90, False), (60, 60, True), (38, 87, True)])
def test_small_and_large_scales_in_every_kernel(ea, eb, least, kind, block, M, N, K):
    """Scales of 2^ea and 2^eb up to twice that.  A block of A in three and one of B in four are zeros, which have the
    quantiser's least scale in A; with `least` all other values are 0 or the least one.  What overflows when its terms' magnitudes
    are added is left out.  Beside the file's bound each block's products and addition lose half of the least fp32 number
    where they are below 2^-126, and slices once more: less than 2^-148 for each."""
    c = Case(M, N, K, kind, kind, "f32", block=block)
    g = torch.Generator(device="cuda").manual_seed(M + N)
    dev = c.A.device
    for s, e in ((c.sa, ea), (c.sb, eb)):
        s.copy_((1 + torch.rand(s.shape, generator=g, device=dev)) * 2.0 ** e)
    for v, n in ((c.A.view(torch.uint8), 3), (c.B.view(torch.uint8), 4)):
        if least:
            v.copy_((torch.rand(v.shape, generator=g, device=dev) < 0.05).to(torch.uint8))
        for j in range(blocks(K)):
            rows = torch.arange(v.shape[0], device=dev) % n == j % n
            v[rows, 128 * j:128 * j + 128] = 0
            if n == 3:
                c.sa[j, rows] = 2.0 ** -126
    c.run()
    torch.cuda.synchronize()
    assert B.gemm_epi_last_error() == B.GE_OK
    got = c.buf[c.at:c.at + M, :N]
    y, mag = c.want()
    on = mag < 2.0 ** 127
    assert bool(on.any()) and bool(got[on].isfinite().all())
    lim = mag * (2.0 ** -16 + (blocks(K) + 4) * 2.0 ** -23) + y.abs() * U["f32"] + (blocks(K) + 4) * 2.0 ** -148
    off = (got.double() - y).abs()
    worst = (off / lim)[on].max().item()
    assert worst <= 1.0, (worst, ((off > lim) & on).nonzero()[:4].tolist())
    B.gemm_epi_fp8_plan_destroy(c.plan)


@pytest.mark.parametrize("kw,status", [
    (dict(M=(1 << 31) - 256), "GE_ERR_SHAPE"), (dict(N=(1 << 31) - 256), "GE_ERR_SHAPE"), (dict(K=(1 << 31) - 256), "GE_ERR_SHAPE"),
    (dict(lda=1 << 31), "GE_ERR_SHAPE"), (dict(ldd=1 << 31), "GE_ERR_SHAPE"),
    (dict(M=(1 << 31) - 257, K=24), "GE_ERR_MISALIGNED"), (dict(N=(1 << 31) - 257, K=24), "GE_ERR_MISALIGNED"),
    (dict(K=(1 << 31) - 257), "GE_ERR_MISALIGNED")])  # (sizes are looked at before pitches)
def test_largest_sizes(kw, status):
    assert bad(**kw) == getattr(B, status)
