"""GPU tests of the fused row quantisers (include/rowquant.h) against their definition
in 64 bits.

Bar, derived from the roundings counted below (u = 2^-24, half a step of fp32):
  * v is an fp32 value within VREL |v| of the definition's.  Norm: the sum of squares is
    a tree of at most 16 * 8 sequential and 6 + 16 joined additions (150 u), halved by
    the square root, and five more roundings: under 80 u < 2^-17.  Gated activation: the
    exponential within 4 u, the reciprocal 2 u, four products and a sum: under 2^-20.
  * codes: |q - v/s| <= half a step of the 8-bit type at v/s + VREL |v/s|; s is checked
    against the definition with the same relative bound and is otherwise taken as given.
  * h is x + residual rounded once to the inputs' type, from an fp32 sum: the bits are
    those of the exact sum rounded to fp32 and then to the type.
"""
import pytest

from gpu_helpers import lib, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
VREL = {"norm": 2.0 ** -17, "swiglu": 2.0 ** -20}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    lib()


def rq():
    from w4a16_dequant_gemm_amd import rowquant
    return rowquant


def rows(T, W, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, W, generator=g) * scale
    x[:, ::97] *= 20.0
    return x.to(DT[dtype]).cuda()


def e4m3_half_step(t):
    e = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(e - 4)


def check(kind, dtype, v, q, s, vrel):
    """v: the definition's values in 64 bits."""
    T, W = v.shape
    if kind == "x16":
        assert s is None and q.dtype == DT[dtype]
        err = (q.double() - v).abs()
        tiny = torch.finfo(DT[dtype]).smallest_normal * torch.finfo(DT[dtype]).eps
        bound = v.abs() * (torch.finfo(DT[dtype]).eps / 2 + vrel) + tiny / 2
        assert bool((err <= bound).all())
        return
    if kind == "int8":
        top = v.abs().amax(1)
        assert bool(((s.double() - top / 127).abs() <= (vrel + 2.0 ** -23) * top / 127).all())
        t = v / torch.where(s > 0, s.double(), 1.0)[:, None]
        assert bool((q.double().abs() <= 127).all())
        assert bool(((q.double() - t).abs() <= 0.5 + (vrel + 2.0 ** -22) * t.abs()).all())
        return
    size = 32 if kind == "mx" else 128
    nb = -(-W // size)
    pad = torch.zeros(T, nb * size, dtype=torch.float64, device=v.device)
    pad[:, :W] = v
    top = pad.view(T, nb, size).abs().amax(-1)
    if kind == "fp8":
        want = top.clamp(min=2.0 ** -110) / 448
        assert bool(((s.double() - want).abs() <= (vrel + 2.0 ** -22) * want).all())
        unit = s.double()
    else:
        # E = floor(log2 top) - 8, either side of a power of two that vrel reaches
        lo = torch.floor(torch.log2((top * (1 - vrel)).clamp(min=2.0 ** -300))) - 8
        hi = torch.floor(torch.log2((top * (1 + vrel)).clamp(min=2.0 ** -300))) - 8
        e = s.double() - 127
        assert bool(((e >= lo.clamp(min=-127)) & (e <= hi.clamp(min=-127))).all())
        unit = torch.exp2(e)
    t = (v / unit.repeat_interleave(size, 1)[:, :W]).clamp(-448, 448)
    got = q.view(torch.float8_e4m3fn).float().double()
    assert bool(((got - t).abs() <= e4m3_half_step(t) + (vrel + 2.0 ** -22) * t.abs()).all())


def norm_values(x, r, w, eps):
    h = x.double() if r is None else x.double() + r.double()
    return h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w.double()


def silu_values(g, u):
    g, u = g.double(), u.double()
    return g * torch.sigmoid(g) * u


KINDS = ["fp8", "int8", "mx", "x16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,W", [(1, 32), (1, 4096), (3, 160), (5, 1024), (4, 1056), (2, 5120),
                                 (7, 8224), (2, 16416), (2, 33024), (1, 131072)])
def test_norm(kind, dtype, T, W):
    for with_r in (False, True):
        say(f"norm {kind} {dtype} T={T} W={W} residual={with_r}")
        x, w = rows(T, W, dtype, 1), (1 + 0.2 * rows(1, W, dtype, 2).float())[0].to(DT[dtype])
        r = rows(T, W, dtype, 3) if with_r else None
        q, s, h = rq().rmsnorm_quantize_rows(x, w, residual=r, eps=1e-5, kind=kind)
        torch.cuda.synchronize()
        check(kind, dtype, norm_values(x, r, w, 1e-5), q, s, VREL["norm"])
        if with_r:
            want = (x.float() + r.float()).to(DT[dtype])
            assert torch.equal(h.view(torch.int16), want.view(torch.int16))
        else:
            assert h is None


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,W", [(1, 32), (1, 128), (3, 160), (9, 1056), (2, 28672), (65, 2848),
                                 (300, 256)])
def test_swiglu_halves_of_one_tensor(kind, dtype, T, W):
    say(f"swiglu {kind} {dtype} T={T} W={W}")
    both = rows(T, 2 * W, dtype, 5)
    gate, up = both[:, :W], both[:, W:]
    q, s = rq().swiglu_quantize_rows(gate, up, kind=kind)
    torch.cuda.synchronize()
    check(kind, dtype, silu_values(gate, up), q, s, VREL["swiglu"])


@pytest.mark.parametrize("W", [16, 48, 144])
def test_widths_of_16(W):
    say(f"widths {W}")
    x, w = rows(5, W, "bf16", 11), torch.ones(W, dtype=torch.bfloat16, device="cuda")
    for kind in ("fp8", "int8", "x16"):
        q, s, _ = rq().rmsnorm_quantize_rows(x, w, kind=kind)
        check(kind, "bf16", norm_values(x, None, w, 1e-6), q, s, VREL["norm"])
        q, s = rq().swiglu_quantize_rows(x, x, kind=kind)
        check(kind, "bf16", silu_values(x, x), q, s, VREL["swiglu"])


@pytest.mark.parametrize("kind", KINDS)
def test_rows_of_zeros_and_single_values(kind):
    say(f"zeros {kind}")
    W = 512
    x = torch.zeros(4, W, dtype=torch.float16, device="cuda")
    x[1, 3] = 2.0
    x[2, 511] = -1.5
    x[3, 128] = 6e-8                                   # the smallest subnormal
    w = torch.ones(W, dtype=torch.float16, device="cuda")
    q, s, _ = rq().rmsnorm_quantize_rows(x, w, eps=1e-6, kind=kind)
    check(kind, "fp16", norm_values(x, None, w, 1e-6), q, s, VREL["norm"])
    q, s = rq().swiglu_quantize_rows(x, x, kind=kind)
    check(kind, "fp16", silu_values(x, x), q, s, VREL["swiglu"])
    assert bool((q.view(torch.uint8)[0] == 0).all()) if kind != "x16" else True


def test_far_gates():
    """Gates where exp overflows or vanishes: silu is g or (nearly) 0, never NaN."""
    g = torch.tensor([-3e38, -1e4, -200.0, -90.0, -87.0, -60.0, -20.0, -1.0, -1e-30, 0.0, 1e-30, 1.0,
                      20.0, 90.0, 1e4, 3e38], dtype=torch.bfloat16, device="cuda")[None]
    u = torch.ones_like(g)
    q, _ = rq().swiglu_quantize_rows(g, u, kind="x16")
    want = silu_values(g, u)
    got = q.double()
    assert bool(torch.isfinite(got).all())
    # below exp(-87) the result may be 0: at most 90 * 2^-126 off
    bound = want.abs() * (2.0 ** -8 + 2.0 ** -20) + 90 * 2.0 ** -126
    assert bool(((got - want).abs() <= bound).all())


@pytest.mark.parametrize("kind", ["fp8", "mx"])
def test_every_code_is_reached_and_ties_go_to_even(kind):
    """Rows whose block maximum makes the scale a power of two: the codes are those of
    torch's own conversion, bit for bit."""
    # gate 64 makes silu(gate) = 64 exactly (1 + exp(-64) is 1 in fp32)
    vals = torch.arange(0, 128, dtype=torch.float32) * (448.0 / 128)
    blocks = torch.stack([vals, -vals, vals / 64, vals / 4096]).repeat(1, 1)
    blocks[:, 0] = 448.0
    u = (blocks.reshape(1, -1)).to(torch.bfloat16).cuda()
    g = torch.full_like(u, 64.0)
    q, s = rq().swiglu_quantize_rows(g, u, kind=kind)
    v = 64.0 * u.float()
    unit = (s.float() if kind == "fp8" else torch.exp2(s.float() - 127))
    unit = unit.repeat_interleave(128 if kind == "fp8" else 32, 1)
    want = (v / unit).to(torch.float8_e4m3fn)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))


def test_strides_do_not_matter():
    T, W = 6, 768
    wide = rows(T, W + 264, "bf16", 21)
    x = wide[:, 8:8 + W]
    r = rows(T, 2 * W, "bf16", 22)[:, W:]
    w = torch.ones(W, dtype=torch.bfloat16, device="cuda")
    for kind in KINDS:
        a = rq().rmsnorm_quantize_rows(x, w, residual=r, kind=kind)
        b = rq().rmsnorm_quantize_rows(x.contiguous(), w, residual=r.contiguous(), kind=kind)
        c = rq().swiglu_quantize_rows(x, r, kind=kind)
        d = rq().swiglu_quantize_rows(x.contiguous(), r.contiguous(), kind=kind)
        for p, o in list(zip(a, b)) + list(zip(c, d)):
            if p is not None:
                assert torch.equal(p.view(torch.uint8), o.view(torch.uint8))


def test_int8_and_mx_rows_equal_the_separate_quantisers():
    """Gate 64 leaves 64 * up exactly; the fused rows are those of the routes' own
    quantisers on that tensor."""
    from w4a16_dequant_gemm_amd import mxfp4, w4a8
    u = rows(9, 1024, "bf16", 31)
    g = torch.full_like(u, 64.0)
    v = (64.0 * u.float()).to(torch.bfloat16)
    q, s = rq().swiglu_quantize_rows(g, u, kind="int8")
    q2, s2 = w4a8.w4a8_quantize_rows(v)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    q, s = rq().swiglu_quantize_rows(g, u, kind="mx")
    q2, s2 = mxfp4.mxfp4_quantize_rows(v)
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_no_rows():
    x = torch.empty(0, 256, dtype=torch.float16, device="cuda")
    w = torch.ones(256, dtype=torch.float16, device="cuda")
    q, s, h = rq().rmsnorm_quantize_rows(x, w, residual=x)
    assert q.shape == (0, 256) and s.shape == (0, 2) and h.shape == (0, 256)
    q, s = rq().swiglu_quantize_rows(x, x, kind="mx")
    assert q.shape == (0, 256) and s.shape == (0, 8)


def test_another_stream_and_a_graph():
    x, r = rows(5, 2048, "bf16", 41), rows(5, 2048, "bf16", 42)
    w = torch.ones(2048, dtype=torch.bfloat16, device="cuda")
    want = rq().rmsnorm_quantize_rows(x, w, residual=r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = rq().rmsnorm_quantize_rows(x, w, residual=r, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    out = tuple(torch.empty_like(t) for t in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rq().rmsnorm_quantize_rows(x, w, residual=r, q=out[0], s=out[1], h=out[2])
    for rep in range(3):
        for t in out:
            t.view(torch.uint8).fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), rep


# Gates beyond which exp(-gate) or the result leaves fp32's normal numbers, and factors that
# bring the result back into them.
FAR = {"fp16": ([-86.9, -87.5, -88.0, -90.0, -95.0, -100.0, -103.0, -104.0, -110.0, -200.0, -1e4,
                 -65504.0, 88.0, 1e4], [1.0, 100.0, 65504.0]),
       "bf16": ([-86.9, -87.5, -88.0, -90.0, -95.0, -100.0, -103.0, -104.0, -110.0, -150.0, -199.0,
                 -200.0, -201.0, -1e4, -3e38, 88.0, 90.0],
                [2.0 ** -100, 1.0, 100.0, 2.0 ** 60, 2.0 ** 100, 2.0 ** 127])}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_far_gates_keep_their_definition(kind, dtype):
    """Whole rows of one far gate, up of one magnitude.  v is an fp32 number: where its own
    value is subnormal it is off by up to a step, 2^-149, and what lies below half of that is 0."""
    W = 256
    gates, ups = FAR[dtype]
    g = torch.tensor(gates, dtype=torch.float64).repeat_interleave(len(ups))[:, None].repeat(1, W)
    gen = torch.Generator().manual_seed(51)
    u = torch.tensor(ups, dtype=torch.float64).repeat(len(gates))[:, None]
    u = u * (0.25 + 0.75 * torch.rand(len(g), W, generator=gen, dtype=torch.float64))
    u *= torch.randint(0, 2, u.shape, generator=gen) * 2 - 1
    g, u = g.to(DT[dtype]).cuda(), u.to(DT[dtype]).cuda()
    v = g.double() / (1 + torch.exp(-g.double())) * u.double()
    keep = v.abs().amax(1) < 3e38                       # results that fp32 holds
    if kind == "x16":
        keep &= v.abs().amax(1) < torch.finfo(DT[dtype]).max
    g, u, v = g[keep], u[keep], v[keep]
    assert len(g) > len(gates)
    say(f"far gates {kind} {dtype}: {len(g)} rows")
    q, s = rq().swiglu_quantize_rows(g, u, kind=kind)
    torch.cuda.synchronize()
    vrel, step = VREL["swiglu"], 2.0 ** -149
    off = vrel * v.abs() + step                         # how far the kernel's v may be off
    if kind == "x16":
        info = torch.finfo(DT[dtype])
        err = (q.double() - v).abs()
        assert bool((err <= off + v.abs() * info.eps / 2 + info.smallest_normal * info.eps / 2).all())
        return
    size = {"fp8": 128, "mx": 32, "int8": W}[kind]
    top = v.abs().view(len(v), -1, size).amax(-1)
    top_off = off.view(len(v), -1, size).amax(-1)
    if kind == "mx":
        lo = torch.floor(torch.log2((top - top_off).clamp(min=2.0 ** -300))) - 8
        hi = torch.floor(torch.log2(top + top_off)) - 8
        e = s.double() - 127
        assert bool(((e >= lo.clamp(min=-127)) & (e <= hi.clamp(min=-127))).all())
        unit = torch.exp2(e)
    else:
        s = s.double().view(len(v), -1)
        want = top.clamp(min=2.0 ** -110) / 448 if kind == "fp8" else top / 127
        # the scale's own rounding, subnormal ones (int8) included
        assert bool(((s - want).abs() <= top_off / 127 + want * 2.0 ** -22 + step).all())
        unit = torch.where(s > 0, s, 1.0)
    unit = unit.repeat_interleave(size, 1)
    t = v / unit
    # what v's error is in codes; the product with 448 / max and its factor's rounding
    slack = off / unit + 2.0 ** -22 * t.abs()
    if kind == "int8":
        t = t.clamp(-127, 127)      # a subnormal scale is rounded so far that v / s passes 127
        assert bool(((q.double() - t).abs() <= 0.5 + slack)[top.repeat_interleave(size, 1) > 0].all())
        zero = v.abs().amax(1) < step / 2 * (1 - vrel)
        assert bool((q[zero] == 0).all()) and bool((s[zero] == 0).all())
        return
    t = t.clamp(-448, 448)
    got = q.view(torch.float8_e4m3fn).float().double()
    assert bool(((got - t).abs() <= e4m3_half_step(t) + slack).all())
    # nothing of a block that vanishes remains
    gone = (top < 2.0 ** -151).repeat_interleave(size, 1)
    assert bool(gone.any()) and bool((got[gone] == 0).all())


def spoil(t, bad):
    """`bad` in row 1 at 0 and 37, row 3 at the end; returns the spoilt elements."""
    where = torch.zeros(t.shape, dtype=torch.bool, device=t.device)
    where[1, 0] = where[1, 37] = where[3, -1] = True
    t[where] = bad
    return where


def shows(kind, q, s, where):
    """Which blocks (rows for int8, elements for x16) hold a spoilt element, and which say so."""
    T, W = where.shape
    if kind == "x16":
        return where, ~torch.isfinite(q.float())
    size = {"fp8": 128, "mx": 32, "int8": W}[kind]
    s = s.view(T, -1)
    return (where.view(T, -1, size).any(-1),
            s == 255 if kind == "mx" else ~torch.isfinite(s))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_what_is_not_finite_shows(kind, dtype, bad):
    T, W = 5, 2304
    say(f"not finite {kind} {dtype} {bad}")
    g, u = rows(T, W, dtype, 61), rows(T, W, dtype, 62)
    clean_q, clean_s = rq().swiglu_quantize_rows(g, u, kind=kind)
    for side in ("gate", "up"):
        g2, u2 = g.clone(), u.clone()
        where = spoil(g2 if side == "gate" else u2, bad)
        q, s = rq().swiglu_quantize_rows(g2, u2, kind=kind)
        want, got = shows(kind, q, s, where)
        assert torch.equal(got, want), side
        size = W // want.shape[1]
        same = ~want.repeat_interleave(size, 1)
        assert torch.equal(q.view(torch.int16 if kind == "x16" else torch.uint8)[same],
                           clean_q.view(torch.int16 if kind == "x16" else torch.uint8)[same])
        if kind != "x16":
            assert torch.equal(s.view(T, -1)[~want], clean_s.view(T, -1)[~want])
    w = torch.ones(W, dtype=DT[dtype], device="cuda")
    clean_q, clean_s, _ = rq().rmsnorm_quantize_rows(g, w, kind=kind)
    g2 = g.clone()
    where = spoil(g2, bad)
    q, s, _ = rq().rmsnorm_quantize_rows(g2, w, kind=kind)
    want, got = shows(kind, q, s, where)
    assert bool(got[want].all())
    clean = torch.tensor([0, 2, 4], device="cuda")
    assert torch.equal(q[clean].view(torch.uint8), clean_q[clean].view(torch.uint8))
    assert not bool(got[clean].any())


@pytest.mark.parametrize("kind", ["fp8", "int8", "mx"])
@pytest.mark.parametrize("rows_", [4, 40])
def test_what_is_not_finite_shows_in_the_product(kind, rows_):
    from w4a16_dequant_gemm_amd import fp8, mxfp4, w4a8
    K, N = 1024, 256
    say(f"not finite through the product {kind} {rows_} rows")
    gen = torch.Generator().manual_seed(63)
    if kind == "fp8":
        w = torch.randint(0, 127, (N, K), generator=gen, dtype=torch.uint8).cuda()
        packed = fp8.fp8_repack(w, torch.full((2, 8), 1e-3, device="cuda"))
        product = lambda q, s: fp8.fp8_gemm(q, s, packed)            # noqa: E731
    else:
        code = torch.randint(-2 ** 31, 2 ** 31 - 1, (K // 8, N), generator=gen).to(torch.int32).cuda()
        if kind == "mx":
            packed = mxfp4.mxfp4_repack(code, torch.full((K // 32, N), 120, dtype=torch.uint8,
                                                         device="cuda"), K, N)
            product = lambda q, s: mxfp4.mxfp4_gemm(q, s, packed, out="bf16")   # noqa: E731
        else:
            one = torch.ones(K // 128, N, dtype=torch.uint8, device="cuda")
            packed = w4a8.w4a8_repack(code, one, one, torch.ones(N, device="cuda"), K, N, 128)
            product = lambda q, s: w4a8.w4a8_gemm(q, s, packed, out="bf16")     # noqa: E731
    g, u = rows(rows_, K, "bf16", 64), rows(rows_, K, "bf16", 65)
    clean = product(*rq().swiglu_quantize_rows(g, u, kind=kind))
    assert bool(torch.isfinite(clean.float()).all())
    for bad in (float("nan"), float("inf")):
        u2 = u.clone()
        u2[2, 700] = bad
        got = product(*rq().swiglu_quantize_rows(g, u2, kind=kind))
        assert not bool(torch.isfinite(got[2].float()).any())
        keep = torch.arange(rows_, device="cuda") != 2
        assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("W", [288, 5120, 33024, 70016])
def test_norm_of_rows_whose_squares_leave_fp32(kind, W):
    """bf16 rows of 2^60 and more have squares beyond fp32, rows of 2^-50 and less squares
    that vanish beside no eps; the norm itself does not."""
    scales = [2.0 ** 60, 2.0 ** 100, 2.0 ** 118, 2.0 ** -50, 2.0 ** -100, 2.0 ** -120, 1.0]
    x = torch.cat([rows(1, W, "bf16", 71 + i) * c for i, c in enumerate(scales)])
    w = (1 + 0.2 * rows(1, W, "bf16", 70).float())[0].to(torch.bfloat16)
    for eps in (0.0, 1e-30, 1e-6):
        say(f"norm of far rows {kind} W={W} eps={eps}")
        for r in (None, x.flip(1) * 0.5):
            q, s, h = rq().rmsnorm_quantize_rows(x, w, residual=r, eps=eps, kind=kind)
            torch.cuda.synchronize()
            check(kind, "bf16", norm_values(x, r, w, eps), q, s, VREL["norm"])
            if r is not None:
                want = (x.float() + r.float()).to(torch.bfloat16)
                assert torch.equal(h.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("kind", ["fp8", "int8", "mx"])
def test_scales_go_to_any_place_in_a_tensor(kind):
    x, u = rows(3, 640, "bf16", 81), rows(3, 640, "bf16", 82)
    w = torch.ones(640, dtype=torch.bfloat16, device="cuda")
    for call in (lambda s: rq().rmsnorm_quantize_rows(x, w, kind=kind, s=s),
                 lambda s: rq().swiglu_quantize_rows(x, u, kind=kind, s=s)):
        want = call(None)
        for shift in (1, 2, 3):
            room = torch.empty(want[1].numel() + 8, dtype=want[1].dtype, device="cuda")
            s = room[shift:shift + want[1].numel()].view(want[1].shape)
            say(f"scales at {s.data_ptr() % 16} of 16, {kind}")
            got = call(s)
            assert torch.equal(s, want[1]) and torch.equal(got[0].view(torch.uint8),
                                                           want[0].view(torch.uint8))


def far_rows(T, W, dtype):
    """Rows that differ from their neighbours, made in place (their number is large)."""
    x = torch.empty(T, W, dtype=DT[dtype], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(91)
    for at in range(0, T, 1 << 26):
        x[at:at + (1 << 26)].normal_(generator=g)
    return x


@pytest.mark.parametrize("kind,dtype", [("int8", "bf16"), ("fp8", "fp16"), ("x16", "bf16")])
def test_norm_of_more_rows_than_one_launch_holds(kind, dtype):
    """64 threads a row: 2^26 rows are 2^32 work-items."""
    T, W, most = (1 << 26) + 5, 16, ((1 << 32) - 1) // 64
    say(f"norm of {T} rows {kind}")
    x, w = far_rows(T, W, dtype), torch.ones(W, dtype=DT[dtype], device="cuda")
    q, s, h = rq().rmsnorm_quantize_rows(x, w, residual=x, kind=kind)
    for at in (slice(0, 100), slice(most - 100, most + 6), slice(T - 100, T)):
        part = x[at].clone()
        want = rq().rmsnorm_quantize_rows(part, w, residual=part, kind=kind)
        for got, ref in zip((q, s, h), want):
            if ref is not None:
                assert torch.equal(got[at].view(torch.uint8), ref.view(torch.uint8)), at


@pytest.mark.parametrize("kind", ["fp8", "x16"])
def test_swiglu_of_more_rows_than_one_launch_holds(kind):
    """8 threads a block of 128: 2^29 rows are 2^32 work-items, and 2^34 bytes."""
    T, W, most = (1 << 29) + 3, 16, ((1 << 32) - 257) // 8
    say(f"swiglu of {T} rows {kind}")
    x = far_rows(T, W, "bf16")
    q, s = rq().swiglu_quantize_rows(x, x, kind=kind)
    for at in (slice(0, 100), slice(most - 100, most + 6), slice(T - 100, T)):
        part = x[at].clone()
        want = rq().swiglu_quantize_rows(part, part, kind=kind)
        for got, ref in zip((q, s), want):
            if ref is not None:
                assert torch.equal(got[at].view(torch.uint8), ref.view(torch.uint8)), at
    del x, q, s
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("W", [32, 2048, 20480, 70016])
def test_norm_in_place(kind, W):
    """h may be x or the residual."""
    x, r = rows(7, W, "bf16", 95), rows(7, W, "bf16", 96)
    w = torch.ones(W, dtype=torch.bfloat16, device="cuda")
    want = rq().rmsnorm_quantize_rows(x, w, residual=r, kind=kind)
    say(f"norm in place {kind} W={W}")
    for side in (0, 1):
        pair = [x.clone(), r.clone()]
        got = rq().rmsnorm_quantize_rows(pair[0], w, residual=pair[1], kind=kind, h=pair[side])
        assert got[2] is pair[side]
        for a, b in zip(got, want):
            assert a is b is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
