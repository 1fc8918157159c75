"""GPU tests of the low-rank adapters (include/lora.h) against their definition in 64 bits.

Bar, derived from the roundings counted below (u = 2^-24, half a step of fp32).  With
S = sum over ranks of |scale| (sum over k |x a|) |b|, the delta is off by at most
  * K + 32 additions of products that are exact (16-bit operands) in the first sum, and for
    E4M3 rows one more product per block, then the scale: (K + 40) u S;
  * the split of h: 2^-18 (bf16), 2^-22 (fp16) of it, fp16 also 2^-38 of the row's largest;
  * 2 R additions in the second sum: 2 R u S (each number counts with its high and low part);
then comes the sum with base, u, and half a step of the output's type.  Matrix instructions may
add the products of a group in any order: every addition is counted, twice for what an
aligning adder drops.
"""
import pytest

from gpu_helpers import lib, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    lib()


def lr():
    from w4a16_dequant_gemm_amd import lora
    return lora


def make_ids(M, L, how, g):
    if how == "one":
        return torch.full((M,), L - 1, dtype=torch.int32)
    if how == "none":
        return torch.full((M,), -1, dtype=torch.int32)
    if how == "mixed":       # neighbours differ, some without an adapter, some out of range
        ids = torch.randint(-1, L, (M,), generator=g).to(torch.int32)
        ids[::13] = L
        ids[5::29] = -(1 << 31)
        ids[7::31] = (1 << 31) - 1
        return ids
    at, ids = 0, torch.empty(M, dtype=torch.int32)      # runs of one request each
    while at < M:
        n = int(torch.randint(1, 60, (1,), generator=g))
        ids[at:at + n] = int(torch.randint(-1, L, (1,), generator=g))
        at += n
    return ids


def problem(M, N, K, R, L, dtype, rows, how, seed=0):
    g = torch.Generator().manual_seed(seed + M + N + K + R)
    t = DT[dtype]
    p = dict(base=torch.randn(M, N, generator=g).to(t), ids=make_ids(M, L, how, g),
             a=(torch.randn(L, R, K, generator=g) * K ** -0.5).to(t),
             b=(torch.randn(L, N, R, generator=g) * R ** -0.5).to(t),
             scale=torch.rand(L, generator=g) * 2 - 0.5, xs=None)
    x = torch.randn(M, K, generator=g)
    if rows == "fp8":
        kb = -(-K // 128)
        p["xs"] = torch.rand(M, kb, generator=g) * 0.01 + 0.001
        p["x"] = (x * 100).clamp(-448, 448).to(E4M3)
    else:
        p["x"] = x.to(t)
    return {k: None if v is None else v.cuda() for k, v in p.items()}


def define(p):
    """(out, S, the row's largest |h| times sum |b|) in 64 bits."""
    x = p["x"].double()
    if p["xs"] is not None:
        x = x * p["xs"].double().repeat_interleave(128, 1)[:, :x.shape[1]]
    out, S, top = p["base"].double(), torch.zeros_like(p["base"], dtype=torch.float64), None
    top = torch.zeros_like(S)
    scale = torch.ones(p["a"].shape[0], dtype=torch.float64) if p["scale"] is None \
        else p["scale"].double()
    for a in range(p["a"].shape[0]):
        m = (p["ids"] == a).nonzero()[:, 0]
        A, B = p["a"][a].double(), p["b"][a].double()
        h = x[m] @ A.t() * scale[a]
        out[m] += h @ B.t()
        S[m] = (x[m].abs() @ A.abs().t() * scale[a].abs()) @ B.abs().t()
        if m.numel():
            top[m] = h.abs().amax(1, keepdim=True) * B.abs().sum(1)
    return out, S, top


def check(got, p, dtype):
    want, S, top = define(p)
    K, R = p["x"].shape[1], p["a"].shape[1]
    part = 2.0 ** -18 if dtype == "bf16" else 2.0 ** -22
    delta = (2 * (K + 40 + 2 * R) * U + part) * S + (2.0 ** -38 * top if dtype == "fp16" else 0.0)
    eps = torch.finfo(DT[dtype]).eps / 2
    tiny = torch.finfo(DT[dtype]).smallest_normal * torch.finfo(DT[dtype]).eps
    bound = delta * (1 + eps) + (eps + 2 * U) * want.abs() + tiny / 2
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    without = (p["ids"] < 0) | (p["ids"] >= p["a"].shape[0])
    assert torch.equal(got[without].view(torch.int16), p["base"][without].view(torch.int16))


# every rank group and its neighbours, single rows, tiles of 16 with a rest, the larger
# tiles of many rows; K inside a step, several parts of K; N inside a run of columns
SHAPES = [(1, 64, 256, 16, 1), (1, 4096, 4096, 16, 8), (1, 1, 16, 8, 1), (3, 7, 48, 8, 2),
          (16, 65, 128, 24, 3), (17, 200, 4112, 32, 5), (33, 129, 144, 40, 4), (64, 1000, 1024, 64, 9),
          (65, 72, 272, 72, 3), (30, 96, 2064, 128, 2), (20, 100, 400, 136, 4), (9, 333, 512, 256, 2),
          (530, 130, 256, 16, 4), (600, 70, 144, 64, 3), (515, 264, 128, 128, 3),
          (520, 66, 160, 200, 2), (1030, 129, 1040, 8, 5), (1100, 80, 272, 32, 7),
          (1027, 64, 400, 96, 3)]


@pytest.mark.parametrize("rows", ["x16", "fp8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K,R,L", SHAPES)
def test_lora(M, N, K, R, L, dtype, rows):
    for how in ("one", "mixed", "runs"):
        say(f"lora M={M} N={N} K={K} R={R} L={L} {dtype} {rows} {how}")
        p = problem(M, N, K, R, L, dtype, rows, how)
        got = lr().lora_add(**p)
        torch.cuda.synchronize()
        check(got, p, dtype)
    p["scale"] = None
    check(lr().lora_add(**p), p, dtype)


# every number of rank operands, with columns of the matrix instruction that hold no row
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("R", [24, 40, 96, 112, 144, 168, 192, 224, 248])
def test_ranks_of_few_rows(R, dtype):
    for how in ("one", "mixed"):
        p = problem(9, 333, 256, R, 2, dtype, "x16", how)
        check(lr().lora_add(**p), p, dtype)


@pytest.mark.parametrize("K", [8, 24, 136, 1032])
def test_widths_of_8(K):
    say(f"K={K}")
    p = problem(21, 50, K, 16, 3, "bf16", "x16", "mixed")
    check(lr().lora_add(**p), p, "bf16")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [40, 1100])
def test_whole_numbers_are_exact(dtype, M):
    """Sums that fp32 and the output hold: the bits are those of the definition."""
    say(f"whole numbers M={M} {dtype}")
    g = torch.Generator().manual_seed(M)
    t, N, K, R, L = DT[dtype], 90, 384, 24, 3

    def whole(*shape):
        return (torch.randint(-1, 2, shape, generator=g)
                * (torch.rand(*shape, generator=g) < 0.1)).to(t).cuda()
    p = dict(base=whole(M, N), x=whole(M, K), a=whole(L, R, K), b=whole(L, N, R), xs=None,
             ids=make_ids(M, L, "mixed", g).cuda(), scale=torch.tensor([1.0, 2.0, -0.5]).cuda())
    want = define(p)[0]
    assert float(want.abs().max()) <= 128
    assert torch.equal(lr().lora_add(**p).double(), want)


@pytest.mark.parametrize("M", [40, 1100])
def test_no_adapter_anywhere(M):
    p = problem(M, 130, 256, 16, 3, "bf16", "x16", "none")
    p["base"][3, 7] = float("nan")
    got = lr().lora_add(**p)
    assert torch.equal(got.view(torch.int16), p["base"].view(torch.int16))


@pytest.mark.parametrize("M", [0, 1, 37, 1100])
def test_in_place(M):
    say(f"in place M={M}")
    p = problem(M, 130, 256, 16, 3, "fp16", "x16", "mixed")
    want = lr().lora_add(**p)
    base = p["base"]
    assert lr().lora_add(**p, out=base) is base and torch.equal(base, want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("first", [0, 1, 8, 11])
def test_slices_of_wider_tensors(first, dtype):
    """Columns of one product's output, rows of x with a stride: what lies beside is kept."""
    say(f"columns from {first} {dtype}")
    M, N, K = 35, 99, 128
    p = problem(M, N, K, 16, 3, dtype, "x16", "mixed")
    want = lr().lora_add(**p)
    wide = torch.full((M, 160), 7.0, dtype=DT[dtype], device="cuda")
    wide[:, first:first + N] = p["base"]
    xw = torch.full((M, 200), float("nan"), dtype=DT[dtype], device="cuda")
    xw[:, 8:8 + K] = p["x"]
    part = wide[:, first:first + N]
    q = dict(p, base=part, x=xw[:, 8:8 + K])
    assert torch.equal(lr().lora_add(**q), want)
    lr().lora_add(**q, out=part)
    assert torch.equal(part, want)
    wide[:, first:first + N] = 7.0
    assert bool((wide == 7.0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [33, 1100])
def test_what_is_not_finite_stays_where_it_is(M, dtype, bad):
    say(f"{bad} M={M} {dtype}")
    p = problem(M, 100, 256, 16, 4, dtype, "x16", "mixed")
    want = lr().lora_add(**p)
    q = dict(p, a=p["a"].clone(), b=p["b"].clone(), x=p["x"].clone())
    q["a"][1, 3, 100] = bad            # adapter 1: its rows
    q["b"][2, 50, 5] = bad             # adapter 2: one column of its rows
    row = int((p["ids"] == 0).nonzero()[1, 0])
    q["x"][row, 9] = bad               # one row
    got = lr().lora_add(**q)
    torch.cuda.synchronize()
    ids = p["ids"]
    hurt = torch.zeros_like(want, dtype=torch.bool)
    hurt[ids == 1] = True
    hurt[ids == 2, 50] = True
    hurt[row] = True
    assert torch.equal(got[~hurt], want[~hurt])
    assert not bool(torch.isfinite(got[hurt]).any())


def test_large_inner_products_in_fp16():
    """x . a beyond 65504, brought back by small b: nothing on the way is fp16 alone."""
    p = problem(20, 64, 512, 16, 2, "fp16", "x16", "mixed")
    p["x"] *= 300
    p["a"] *= 3000
    p["b"] *= 2.0 ** -18
    assert float(define(p)[2].max()) > 0
    got = lr().lora_add(**p)
    assert bool(torch.isfinite(got).all())
    # b is a number of 2^-24 steps here; the definition sees the same ones
    check(got, p, "fp16")
    p["x"] *= 2.0 ** -14               # and very small ones
    p["a"] *= 2.0 ** -10
    p["b"] *= 2.0 ** 14
    p["base"].zero_()
    check(lr().lora_add(**p), p, "fp16")


@pytest.mark.parametrize("M", [40, 1100])
def test_a_row_depends_on_itself_alone(M):
    """The same row among others with other adapters, and again: the same bits."""
    p = problem(M, 130, 1040, 24, 5, "bf16", "x16", "one")
    want = lr().lora_add(**p)
    assert torch.equal(lr().lora_add(**p), want)
    q = dict(p, ids=p["ids"].clone())
    q["ids"][1::2] = torch.randint(-1, 5, (M // 2,), dtype=torch.int32).cuda()
    same = q["ids"] == p["ids"]
    assert torch.equal(lr().lora_add(**q)[same], want[same])


def test_offsets_beyond_32_bits():
    """Outputs and adapters of more than 4 GiB each."""
    M, N, K, R, L = 70000, 32768, 16, 8, 2
    say(f"lora M={M} N={N}")
    p = dict(base=torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"), xs=None,
             x=torch.zeros(M, K, dtype=torch.bfloat16, device="cuda"),
             a=torch.ones(L, R, K, dtype=torch.bfloat16, device="cuda"),
             b=torch.ones(L, N, R, dtype=torch.bfloat16, device="cuda"),
             scale=torch.ones(L, device="cuda"),
             ids=torch.full((M,), -1, dtype=torch.int32, device="cuda"))
    p["x"][-1, 0] = p["x"][-3, 1] = 1.0
    p["ids"][-3:] = 1
    lr().lora_add(**p, out=p["base"])
    assert bool((p["base"][-1] == 8).all()) and bool((p["base"][-3] == 8).all())
    assert bool((p["base"][-2] == 0).all()) and int(p["base"].count_nonzero()) == 2 * N
    L, N, R = 600, 16384, 256          # b of 5 GiB
    say(f"lora L={L} N={N} R={R}")
    b = torch.zeros(L, N, R, dtype=torch.bfloat16, device="cuda")
    b[-1, -1, -1] = 1.0
    a = torch.ones(L, R, 16, dtype=torch.bfloat16, device="cuda")
    out = lr().lora_add(torch.zeros(2, N, dtype=torch.bfloat16, device="cuda"),
                        torch.ones(2, 16, dtype=torch.bfloat16, device="cuda"), a, b,
                        torch.tensor([L - 1, L - 2], dtype=torch.int32, device="cuda"))
    assert float(out[0, -1]) == 16.0 and int(out.count_nonzero()) == 1


# the most columns there may be: the grid's second dimension is at its largest
@pytest.mark.parametrize("M", [1, 128])
def test_most_columns(M):
    N, K, R = (1 << 24) - 1, 16, 8
    g = torch.Generator("cuda").manual_seed(M)
    p = dict(base=torch.randn(M, N, generator=g, device="cuda", dtype=torch.bfloat16),
             x=torch.randn(M, K, generator=g, device="cuda").bfloat16(),
             a=torch.randn(1, R, K, generator=g, device="cuda").bfloat16(),
             b=torch.randn(1, N, R, generator=g, device="cuda").bfloat16(),
             ids=torch.zeros(M, dtype=torch.int32, device="cuda"), scale=None, xs=None)
    p["ids"][3::7] = -1
    got = lr().lora_add(**p)
    for first in (0, N // 2 - 7, (N // 4096) * 4096 - 600, N - 1000):
        n = slice(first, first + 1000)
        part = dict(p, base=p["base"][:, n].contiguous(), b=p["b"][:, n].contiguous())
        check(got[:, n].contiguous(), part, "bf16")


def test_on_another_stream():
    p = problem(300, 512, 1024, 16, 4, "bf16", "x16", "runs")
    want = lr().lora_add(**p).cpu()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    big = torch.rand(4096, 4096, device="cuda")
    for _ in range(20):
        big = big @ big * 1e-3
    got = lr().lora_add(**p, stream=side)
    side.synchronize()
    assert torch.equal(got.cpu(), want)
    torch.cuda.synchronize()


def test_graphs_that_run_beside_each_other():
    """Two graphs captured one after the other, replayed on two streams with eager calls on a
    third: no memory between the two products is shared."""
    say("graphs beside each other")
    made = []
    for i, (M, K) in enumerate(((48, 8192), (700, 4096))):
        p = problem(M, 1024, K, 16, 4, "bf16", "x16", "mixed", seed=i)
        want = lr().lora_add(**p)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = lr().lora_add(**p)
        made.append((graph, out, want, p, torch.cuda.Stream()))
    for rep in range(5):
        for graph, out, *_ in made:
            out.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            for graph, _, _, _, stream in made:
                with torch.cuda.stream(stream):
                    graph.replay()
        eager = [lr().lora_add(**m[3]) for m in made]
        torch.cuda.synchronize()
        for (_, out, want, _, _), e in zip(made, eager):
            assert torch.equal(out, want) and torch.equal(e, want), rep


def test_beside_the_products():
    """Next to the 4-bit product and, from the same quantised rows, next to the fp8 product."""
    import w4a16_synth as synth
    from gpu_helpers import OnDevice
    from w4a16_dequant_gemm_amd import fp8, rowquant
    say("beside the products")
    for dtype in ("fp16", "bf16"):
        d = OnDevice(synth.make_problem(20, 512, 256, G=128, dtype=dtype, sym=False, seed=4))
        p = problem(20, 256, 512, 16, 3, dtype, "x16", "mixed")
        p["x"], p["base"] = d.X, d.gemm()
        check(lr().lora_add(**p), p, dtype)
    x = torch.randn(20, 512).to(torch.bfloat16).cuda()
    q, s, _ = rowquant.rmsnorm_quantize_rows(x, torch.ones(512, dtype=torch.bfloat16).cuda())
    w = (torch.randn(256, 512) * 100).clamp(-448, 448).to(E4M3).cuda()
    p = problem(20, 256, 512, 16, 3, "bf16", "fp8", "mixed")
    p["x"], p["xs"] = q, s
    p["base"] = fp8.fp8_gemm(q, s, fp8.fp8_repack(w, torch.full((2, 4), 1e-3).cuda()))
    check(lr().lora_add(**p), p, "bf16")
