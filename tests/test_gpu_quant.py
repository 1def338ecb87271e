"""8-bit values and scales for blocks of 128, against the definition.

The scale is one correctly rounded fp32 division, its inverse another, and a value one fp32 product rounded to
8 bits: all of it can be repeated bit for bit on the CPU.  Against 64 bits a value is off by half a step of
its type, u = finfo.eps / 2 of itself or half of the smallest subnormal, and by the roundings of inverse and product, 2^-23.
"""
import pytest
import torch

from dense_gemm_elementwise_gb300 import build as gbuild

gbuild.build()
from dense_gemm_elementwise_gb300 import binding as B  # noqa: E402

TYPE = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn,
        "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
U = {"e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
LEAST = {"e4m3": 2.0 ** -9, "e5m2": 2.0 ** -16}
SENT = 0xA5


def blocks(n):
    return -(-n // 128)


def up(n, m):
    return -(-n // m) * m


def reference(x, kind, square):
    """(values as bytes, scales) of x (T, D) in fp32, on the CPU."""
    T, D = x.shape
    x = x.float()
    p = torch.nn.functional.pad(x, (0, -D % 128, 0, -T % 128)).abs()
    four = p.reshape(blocks(T), 128, blocks(D), 128)
    four = torch.where(four.isnan(), torch.zeros(()), four)  # NaN is no maximum
    if square:
        amax = four.amax((1, 3))
    else:
        amax = four.amax(3).reshape(-1, blocks(D))[:T]
    scale = (amax / LARGEST[kind]).clamp_min(2.0 ** -126)
    inv = 1 / scale
    wide = inv.repeat_interleave(128, 1)[:, :D]
    if square:
        wide = wide.repeat_interleave(128, 0)[:T]
    q = (x * wide).clamp(-LARGEST[kind], LARGEST[kind]).to(TYPE[kind])
    return q.view(torch.uint8), scale.t().contiguous()


class Case:
    def __init__(self, x, kind="e4m3", block="row", pad=0, extra=0):
        """x: a CPU tensor of the input's type; pad: more elements between its rows; extra: more in every output's pitch."""
        T, D = x.shape
        self.T, self.D, self.kind, self.square = T, D, kind, block == "square"
        dev = torch.device("cuda", 0)
        name = {v: k for k, v in TYPE.items()}[x.dtype]
        self.x_host = x
        self.x = torch.full((T, D + pad), float("nan"), dtype=x.dtype, device=dev)[:, :D]
        self.x.copy_(x)
        self.ldq, self.ldqt = up(D, 16) + 16 * extra, up(T, 16) + 16 * extra
        self.lds = (blocks(T) if self.square else T) + 3 * extra
        self.ldst = (blocks(D) if self.square else D) + 3 * extra
        self.desc = B.make_quant_desc(name, kind, block=block, ldx=D + pad, ldq=self.ldq, ldqt=self.ldqt, lds=self.lds,
                                      ldst=self.ldst)
        self.plan = B.gemm_epi_quant_plan_create(T, D, self.desc)
        self.q = torch.full((T + 2, self.ldq), SENT, dtype=torch.uint8, device=dev)
        self.qt = torch.full((D + 2, self.ldqt), SENT, dtype=torch.uint8, device=dev)
        self.scale = torch.full((blocks(D) + 1, self.lds), -7.0, device=dev)
        self.scale_t = torch.full((blocks(T) + 1, self.ldst), -7.0, device=dev)

    def run(self, rows=True, cols=True, stream=None):
        B.gemm_epi_quant_run(self.plan, self.x, self.q if rows else None, self.scale if rows else None,
                             self.qt if cols else None, self.scale_t if cols else None, stream=stream)
        return self

    def check(self, rows=True, cols=True):
        torch.cuda.synchronize()
        for on, q, s, x in ((rows, self.q, self.scale, self.x_host), (cols, self.qt, self.scale_t, self.x_host.t())):
            q, s = q.cpu(), s.cpu()
            if not on:
                assert bool((q == SENT).all()) and bool((s == -7.0).all())
                continue
            n, k = x.shape
            want, scale = reference(x, self.kind, self.square)
            ns = scale.shape[1]
            assert torch.equal(s[:-1, :ns], scale)
            same = q[:n, :k] == want
            nan = want.view(TYPE[self.kind]).float().isnan()  # either sign of it
            same |= nan & q[:n, :k].contiguous().view(TYPE[self.kind]).float().isnan()
            assert bool(same.all()), (~same).nonzero()[:5]
            # nothing else is written
            assert bool((q[n:] == SENT).all()) and bool((q[:n, k:] == SENT).all())
            assert bool((s[-1] == -7.0).all()) and bool((s[:, ns:] == -7.0).all())
            # and against 64 bits
            fine = x.double().isfinite() & (scale.double().t().repeat_interleave(128, 1)[:, :k] < float("inf") if not self.square else
                                            torch.ones_like(x, dtype=torch.bool))
            wide = scale.double().t().repeat_interleave(128, 1)[:, :k]
            if self.square:
                wide = wide.repeat_interleave(128, 0)[:n]
            fine &= wide < float("inf")
            off = (q[:n, :k].contiguous().view(TYPE[self.kind]).double() * wide - x.double()).abs()
            lim = x.double().abs() * (U[self.kind] + 2.0 ** -22) + wide * LEAST[self.kind] / 2
            assert bool((off <= lim)[fine].all())
        B.gemm_epi_quant_plan_destroy(self.plan)


def some(T, D, x="bf16", seed=0):
    g = torch.Generator().manual_seed(seed + 31 * T + D)
    v = torch.randn(T, D, generator=g) * torch.randn(T, 1, generator=g).exp() * torch.randn(1, D, generator=g).exp()
    return v.clamp(-6e4, 6e4).to(TYPE[x])


@pytest.mark.gpu
@pytest.mark.parametrize("T,D", [(1, 1), (1, 128), (1, 4096), (3, 130), (127, 129), (128, 128), (129, 8), (300, 517), (1025, 72),
                                 (2, 7), (256, 1000)])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block", ["row", "square"])
def test_sizes(T, D, x, block):
    Case(some(T, D, x), block=block).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", ["row", "square"])
@pytest.mark.parametrize("rows,cols", [(True, False), (False, True), (True, True)])
def test_one_output_or_both(kind, block, rows, cols):
    Case(some(200, 390), kind, block, pad=2, extra=1).run(rows, cols).check(rows, cols)


@pytest.mark.gpu
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [1, 4, 8])
def test_pitches(x, pad):
    Case(some(140, 264, x), pad=pad, extra=2).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("block", ["row", "square"])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_zeros_tiny_and_huge_values(block, kind):
    x = some(300, 400, "f32")
    x[:140, :130] = 0.0                      # whole blocks of zeros, either way
    x[140, :] = 1e-44                        # subnormal: the scale's lower limit
    x[150, :] = torch.linspace(-1e-36, 1e-36, 400)
    x[160, :] *= 1e30
    Case(x, kind, block).run().check()


@pytest.mark.gpu
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block", ["row", "square"])
def test_nan_stays_at_its_place_and_infinity_in_its_block(x, block):
    v = some(260, 300, x)
    v[5, 7] = float("nan")
    v[130, 140] = float("inf")
    v[131, 299] = float("-inf")
    Case(v, block=block).run().check()


@pytest.mark.gpu
def test_another_stream_a_graph_and_the_same_bits():
    c = Case(some(333, 520))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.run(stream=s)
    torch.cuda.synchronize()
    first = c.q.clone(), c.qt.clone(), c.scale.clone(), c.scale_t.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(stream=torch.cuda.current_stream())
    for t in (c.q, c.qt):
        t.fill_(SENT)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (c.q, c.qt, c.scale, c.scale_t)):
        assert torch.equal(a, b)
    c.x_host = some(333, 520, seed=9)
    c.x.copy_(c.x_host)
    graph.replay()
    c.check()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    T, D = 34000, 65536  # 2.2e9 elements
    dev = torch.device("cuda", 0)
    x = torch.zeros(T, D, dtype=torch.bfloat16, device=dev)
    tail = some(130, 200)
    x[-130:, -200:] = tail.to(dev)
    plan = B.gemm_epi_quant_plan_create(T, D, B.make_quant_desc("bf16", "e4m3", ldqt=up(T, 16)))
    q, qt = torch.empty(T, D, dtype=torch.uint8, device=dev), torch.empty(D, up(T, 16), dtype=torch.uint8, device=dev)
    s, st = torch.empty(blocks(D), T, device=dev), torch.empty(blocks(T), D, device=dev)
    B.gemm_epi_quant_run(plan, x, q, s, qt, st)
    torch.cuda.synchronize()
    wide = torch.zeros(256, 256, dtype=torch.bfloat16)
    wide[-130:, -200:] = tail
    wq, ws = reference(wide, "e4m3", False)
    assert torch.equal(q[-256:, -256:].cpu(), wq) and torch.equal(s[-2:, -256:].cpu(), ws)
    # T is no multiple of 128: the last column block has 80 rows
    last = T % 128
    wq, ws = reference(wide[-last:].t().contiguous(), "e4m3", False)
    assert torch.equal(qt[-256:, T - last:T].cpu(), wq) and torch.equal(st[-1:, -256:].cpu(), ws)
    B.gemm_epi_quant_plan_destroy(plan)


def bad(T=100, D=64, x="bf16", q="e4m3", **kw):
    reserved = kw.pop("reserved", 0)
    d = B.make_quant_desc(x, q, **kw)
    d.reserved = reserved
    with pytest.raises(B.GemmEpiError) as e:
        B.gemm_epi_quant_plan_create(T, D, d)
    return e.value.status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), "GE_ERR_SHAPE"), (dict(D=-1), "GE_ERR_SHAPE"), (dict(T=1 << 31), "GE_ERR_SHAPE"),
    (dict(x="e4m3"), "GE_ERR_UNSUPPORTED"), (dict(q="bf16"), "GE_ERR_UNSUPPORTED"), (dict(x=9), "GE_ERR_UNSUPPORTED"),
    (dict(block=2), "GE_ERR_INVALID"), (dict(reserved=1), "GE_ERR_INVALID"), (dict(ldx=63), "GE_ERR_SHAPE"),
    (dict(ldq=72), "GE_ERR_MISALIGNED"), (dict(ldqt=104), "GE_ERR_MISALIGNED"), (dict(ldq=48), "GE_ERR_SHAPE"),
    (dict(lds=99), "GE_ERR_SHAPE"), (dict(ldst=63), "GE_ERR_SHAPE")])
def test_plan_refusals(kw, status):
    assert bad(**kw) == getattr(B, status)


def test_null_plans():
    assert B.lib.gemm_epi_quant_plan_create(None, 1, 1, None) == B.GE_ERR_INVALID
    assert B.lib.gemm_epi_quant_run(None, None, None, None, None, None, None) == B.GE_ERR_INVALID
    B.gemm_epi_quant_plan_destroy(None)


@pytest.mark.gpu
def test_run_refusals():
    c = Case(some(100, 64))
    run = lambda *a: B.gemm_epi_quant_run(c.plan, *a, check=False)  # noqa: E731
    assert run(None, c.q, c.scale, None, None) == B.GE_ERR_MISSING_ARG
    assert run(c.x, None, None, None, None) == B.GE_ERR_MISSING_ARG
    assert run(c.x, c.q, None, None, None) == B.GE_ERR_MISSING_ARG
    assert run(c.x, c.q, c.scale, c.qt, None) == B.GE_ERR_MISSING_ARG
    assert run(c.x, c.q, c.scale, c.q, c.scale_t) == B.GE_ERR_INVALID
    assert run(c.x, c.q, c.scale, c.qt, c.scale) == B.GE_ERR_INVALID
    assert run(c.x.data_ptr() + 2, c.q, c.scale, None, None) == B.GE_ERR_MISALIGNED
    assert run(c.x, c.q.data_ptr() + 8, c.scale, None, None) == B.GE_ERR_MISALIGNED
    # a default pitch that is no whole 16 bytes, of the output that is asked for
    plan = B.gemm_epi_quant_plan_create(100, 64, B.make_quant_desc("bf16", "e4m3"))
    assert B.gemm_epi_quant_run(plan, c.x, None, None, c.qt, c.scale_t, check=False) == B.GE_ERR_MISALIGNED
    assert B.gemm_epi_quant_run(plan, c.x, c.q, c.scale, check=False) == B.GE_OK
    torch.cuda.synchronize()
    B.gemm_epi_quant_plan_destroy(plan)


@pytest.mark.parametrize("kw", [dict(ldx=1 << 31), dict(ldq=1 << 31), dict(ldqt=1 << 31), dict(lds=1 << 31), dict(ldst=1 << 31),
                                dict(T=(1 << 31) - 1, D=1 << 15)])
def test_largest_sizes_and_pitches(kw):
    assert bad(**kw) == B.GE_ERR_SHAPE


@pytest.mark.gpu
@pytest.mark.parametrize("block", ["row", "square"])
def test_the_widest_rows(block):
    """Numbers of columns next to 2^31, of which all but the last 368 and 383 are zeros."""
    dev = torch.device("cuda", 0)

    def wide(D, n, **kw):
        x = torch.zeros(2, D, dtype=torch.bfloat16, device=dev)
        tail = some(2, n)
        x[:, -n:] = tail.to(dev)
        return x, tail, B.gemm_epi_quant_plan_create(2, D, B.make_quant_desc("bf16", "e4m3", block=block, **kw))

    D, n = (1 << 31) - 16, 368
    x, tail, plan = wide(D, n)
    q = torch.full((2, D), SENT, dtype=torch.uint8, device=dev)
    s = torch.full((blocks(D), 1 if block == "square" else 2), -7.0, device=dev)
    B.gemm_epi_quant_run(plan, x, q, s)
    torch.cuda.synchronize()
    B.gemm_epi_quant_plan_destroy(plan)
    wq, ws = reference(tail, "e4m3", block == "square")
    assert torch.equal(q[:, -n:].cpu(), wq) and torch.equal(s[-3:].cpu(), ws)
    assert not bool(q[:, :-n].any()) and bool((s[:-3] == 2.0 ** -126).all())
    del x, q, s
    D, n = (1 << 31) - 1, 383
    x, tail, plan = wide(D, n, ldqt=16)
    qt = torch.full((D + 1, 16), SENT, dtype=torch.uint8, device=dev)
    st = torch.full((1, blocks(D) if block == "square" else D), -7.0, device=dev)
    B.gemm_epi_quant_run(plan, x, None, None, qt, st)
    torch.cuda.synchronize()
    B.gemm_epi_quant_plan_destroy(plan)
    wq, ws = reference(tail.t().contiguous(), "e4m3", block == "square")
    m = ws.shape[1]
    assert torch.equal(qt[-n - 1:-1, :2].cpu(), wq) and torch.equal(st[:, -m:].cpu(), ws)
    assert bool((st[:, :-m] == 2.0 ** -126).all()) and bool((qt[-1] == SENT).all()) and bool((qt[-n:, 2:] == SENT).all())
    assert not bool(qt[:1 << 20, :2].any()) and not bool(qt[-1 << 20:-n - 1, :2].any())
