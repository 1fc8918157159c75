"""GPU tests of the low-rank adapters (include/lora.h): numbers at the ends of the types, and the
forms that their plans take for certain sizes, against the definition in 64 bits."""
import pytest

from gpu_helpers import lib, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    lib()


def lr():
    from w4a16_dequant_gemm_amd import lora
    return lora


# few rows, ordered rows, and both forms for many rows; ranks that fill an operand and not
FORMS = [(3, 16), (3, 40), (200, 40), (600, 64), (600, 40), (1100, 24)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,R", FORMS)
def test_infinite_scale(M, R, dtype):
    """All numbers of h and b are positive: infinite is what comes out, whatever lies behind the
    last rank; other adapters' rows are not touched by it."""
    say(f"infinite scale M={M} R={R} {dtype}")
    N, K = 200, 64
    x = torch.full((M, K), 0.5, dtype=DT[dtype]).cuda()
    a = torch.full((2, R, K), 0.25, dtype=DT[dtype]).cuda()
    b = torch.full((2, N, R), 0.125, dtype=DT[dtype]).cuda()
    base = torch.ones(M, N, dtype=DT[dtype]).cuda()
    ids = (torch.arange(M) % 2).to(torch.int32).cuda()
    out = lr().lora_add(base, x, a, b, ids, scale=torch.tensor([INF, 1.0]).cuda())
    assert bool((out[ids == 0] == INF).all())
    assert bool((out[ids == 1] == 1.0 + R).all())      # 64 / 8 / 8 ranks of one each


@pytest.mark.parametrize("M,R", FORMS)
def test_infinite_rank_beside_large_ones_fp16(M, R):
    """One inner product is infinite, the others lie beyond fp16: an infinity comes out, since
    all of b is positive; where b's number for that rank is zero, NaN, as by the definition."""
    say(f"infinite rank M={M} R={R}")
    N, K = 200, 64
    x = torch.full((M, K), 256.0, dtype=torch.float16).cuda()
    a = torch.full((1, R, K), 128.0, dtype=torch.float16)
    a[0, R // 2, 5] = INF
    b = torch.full((1, N, R), 0.5, dtype=torch.float16)
    b[0, 77, R // 2] = 0.0
    out = lr().lora_add(torch.ones(M, N, dtype=torch.float16).cuda(), x, a.cuda(), b.cuda(),
                        torch.zeros(M, dtype=torch.int32).cuda())
    rest = torch.arange(N) != 77
    assert bool((out[:, rest.cuda()] == INF).all())
    assert bool(torch.isnan(out[:, 77]).all())


@pytest.mark.parametrize("M,R", FORMS)
def test_inner_products_of_24_bits_bf16(M, R):
    """Pairs of ranks whose inner products are whole numbers below 2^24 that share their upper 16
    bits, added and taken away by b: every step is exact in fp32, and what is left are the
    lower 8 bits."""
    say(f"inner products of 24 bits M={M} R={R}")
    N, K = 200, 64
    g = torch.Generator().manual_seed(M + R)
    x = torch.zeros(M, K)
    x[:, 3], x[:, 9], x[:, 40] = 2.0 ** 16, 2.0 ** 8, 1.0
    parts = torch.randint(1, 256, (2, R // 2, 3), generator=g)
    a = torch.zeros(2, R, K)
    a[:, 0::2, 3] = a[:, 1::2, 3] = parts[..., 0].float()
    a[:, 0::2, 9] = a[:, 1::2, 9] = parts[..., 1].float()
    a[:, 0::2, 40] = parts[..., 2].float()
    pair = torch.arange(N) % (R // 2)
    b = torch.zeros(2, N, R)
    b[:, torch.arange(N), 2 * pair] = 1.0
    b[:, torch.arange(N), 2 * pair + 1] = -1.0
    ids = torch.arange(M) % 3 % 2
    out = lr().lora_add(*(t.to(torch.bfloat16).cuda() for t in (torch.zeros(M, N), x, a, b)),
                        ids.to(torch.int32).cuda()).cpu()
    assert torch.equal(out.float(), parts[ids][:, pair, 2].float())


@pytest.mark.parametrize("M,R", FORMS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_inner_products_beyond_bf16(M, R, sign):
    """Inner products between bf16's largest number and fp32's, brought back by b: the definition's
    outputs are ordinary numbers."""
    say(f"inner products beyond bf16 M={M} R={R} sign={sign}")
    N, K = 200, 64
    x, a = torch.zeros(M, K), torch.zeros(1, R, K)
    x[:, 1], a[:, :, 1] = sign * 1.9921875 * 2.0 ** 63, 1.9921875 * 2.0 ** 63
    x[:, 5], a[:, :, 5] = sign * 2.0 ** 63, 1.5 * 2.0 ** 57
    b = torch.zeros(1, N, R)
    b[0, torch.arange(N), torch.arange(N) % R] = 2.0 ** -100
    x, a, b = (t.to(torch.bfloat16) for t in (x, a, b))
    h = x.double() @ a[0].double().t()
    assert 3.3961e38 < float(h.abs().max()) < 3.4028e38
    out = lr().lora_add(torch.zeros(M, N, dtype=torch.bfloat16).cuda(), x.cuda(), a.cuda(),
                        b.cuda(), torch.zeros(M, dtype=torch.int32).cuda()).cpu()
    want = h @ b[0].double().t()
    assert bool(((out.double() - want).abs() <= 2.0 ** -8 * (1 + 2.0 ** -20) * want.abs()).all())


# ---- forms that the plans take for certain sizes
#
# Bar, as at the head of test_gpu_lora.py, with U = 2^-24 and S = sum over ranks of |scale| (sum
# over k |x a|) |b|: K + 40 steps of fp32 in the first sum and its joins, 3 R (bf16: every part of
# a number counts) or 2 R (fp16) in the second, each counted twice; fp16 also 2^-22 of S and
# 2^-38 of the row's largest for what two parts leave out; then half a step of the output.

U = 2.0 ** -24


def check(got, p, dtype):
    want, S, top = define(p)
    K, R = p["x"].shape[1], p["a"].shape[1]
    if dtype == "bf16":
        delta = 2 * (K + 40 + 3 * R) * U * S
    else:
        delta = (2 * (K + 40 + 2 * R) * U + 2.0 ** -22) * S + 2.0 ** -38 * top
    f = torch.finfo(DT[dtype])
    bound = delta * (1 + f.eps / 2) + (f.eps / 2 + 2 * U) * want.abs() \
        + f.smallest_normal * f.eps / 2
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    without = (p["ids"] < 0) | (p["ids"] >= p["a"].shape[0])
    assert torch.equal(got[without].view(torch.int16), p["base"][without].view(torch.int16))


def define(p):
    """(out, S, the row's largest |h| times sum |b|) in 64 bits, over the adapters that are used."""
    x = p["x"].double()
    if p["xs"] is not None:
        x = x * p["xs"].double().repeat_interleave(128, 1)[:, :x.shape[1]]
    out = p["base"].double()
    S, top = torch.zeros_like(out), torch.zeros_like(out)
    for a in p["ids"].unique().tolist():
        if not 0 <= a < p["a"].shape[0]:
            continue
        m = (p["ids"] == a).nonzero()[:, 0]
        A, B, scale = p["a"][a].double(), p["b"][a].double(), p["scale"][a].double()
        h = x[m] @ A.t() * scale
        out[m] += h @ B.t()
        S[m] = (x[m].abs() @ A.abs().t() * scale.abs()) @ B.abs().t()
        top[m] = h.abs().amax(1, keepdim=True) * B.abs().sum(1)
    return out, S, top


def problem(M, N, K, R, L, dtype, rows, ids):
    t, g = DT[dtype], torch.Generator(device="cuda")
    g.manual_seed(M + N + K + R + L)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    x, xs = randn(M, K), None
    if rows == "fp8":
        xs = torch.rand(M, -(-K // 128), generator=g, device="cuda") * 0.01 + 0.001
        x = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    else:
        x = x.to(t)
    return dict(base=randn(M, N).to(t), x=x, xs=xs, ids=ids.to(torch.int32).cuda(),
                a=(randn(L, R, K) * K ** -0.5).to(t), b=(randn(L, N, R) * R ** -0.5).to(t),
                scale=torch.rand(L, generator=g, device="cuda") * 2 - 0.5)


def splits_of(M, N, K, R, L):
    """Parts of K in the plan for many rows, from the workspace that it asks for."""
    places = (M // 64 + L + 1) * 64 if 1 < L <= 64 else M
    fixed = places * ((R + 31) // 32 * 128 + 4 + (8 if L > 1 else 0))
    parts = (lr().lora_workspace_bytes(M, N, K, R, L, 0) - 65536 - fixed) / (places * R * 4)
    assert parts == int(parts)
    return int(parts)


# (shape, parts of K): first products whose loads run on past the first stages, joins of four
# parts and more, second products of 1 to 5 runs of columns a workgroup with whole and
# ragged ends, and every number of operands of 32 ranks
MANY = [((1030, 4200, 8208, 64, 3), 11), ((1030, 9000, 8208, 64, 3), 11),
        ((3000, 9000, 2064, 64, 3), 5), ((3000, 5130, 1040, 64, 3), 3),
        ((2000, 20000, 528, 64, 2), 2), ((2100, 19968, 528, 16, 1), 2),
        ((600, 1000, 8208, 136, 3), 7), ((600, 1000, 4112, 168, 3), 6),
        ((600, 3001, 4112, 256, 3), 5), ((600, 500, 4112, 112, 2), 9)]


@pytest.mark.parametrize("rows", ["x16", "fp8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("shape,splits", MANY)
def test_many_rows(shape, splits, dtype, rows):
    M, N, K, R, L = shape
    say(f"many rows M={M} N={N} K={K} R={R} L={L} {dtype} {rows}")
    assert splits_of(*shape) == splits
    ids = torch.arange(M) // 37 % (L + 1) - 1 if L > 1 else torch.zeros(M)
    p = problem(M, N, K, R, L, dtype, rows, ids)
    check(lr().lora_add(**p), p, dtype)


# more adapters than groups are made for: ordered rows of several adapters in a group, in both
# forms for many rows and in the one for few; above 1023 they share bins of the order
MIXED = [(600, 400, 1040, 64, 100), (600, 401, 1040, 64, 1500), (4000, 130, 528, 24, 100),
         (600, 400, 1040, 16, 1500), (200, 130, 2064, 40, 66), (130, 1000, 144, 16, 100),
         (520, 70, 48, 200, 1100)]


@pytest.mark.parametrize("rows", ["x16", "fp8"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K,R,L", MIXED)
def test_many_adapters(M, N, K, R, L, dtype, rows):
    g = torch.Generator().manual_seed(M + L)
    for how in ("random", "colliding"):
        say(f"many adapters M={M} N={N} K={K} R={R} L={L} {dtype} {rows} {how}")
        ids = torch.randint(-1, L, (M,), generator=g)
        if how == "colliding":     # few remainders of 1023, several adapters each
            ids = torch.tensor([i for i in (0, 1023, 5, 1028, 64, 65, -1) if i < L])[
                torch.randint(0, 100, (M,), generator=g) % (7 if L > 1028 else 5)]
        ids[::17] = L + 5
        p = problem(M, N, K, R, L, dtype, rows, ids)
        got = lr().lora_add(**p)
        check(got, p, dtype)
        base = p["base"]
        p["base"] = base.clone()
        assert torch.equal(lr().lora_add(**p, out=p["base"]), got)


# more rows than the order keeps in registers; one adapter, whose rows are not ordered, with
# groups of rows that have none
@pytest.mark.parametrize("rows", ["x16", "fp8"])
@pytest.mark.parametrize("M,N,K,R,L", [(9300, 70, 48, 16, 40), (9300, 70, 48, 40, 1500),
                                       (20000, 9, 16, 8, 300), (600, 300, 272, 64, 1),
                                       (1100, 300, 272, 16, 1), (300, 300, 272, 64, 1)])
def test_order_of_many_rows_and_none(M, N, K, R, L, rows):
    say(f"order M={M} N={N} K={K} R={R} L={L} {rows}")
    g = torch.Generator().manual_seed(M)
    ids = torch.randint(-1, L, (M,), generator=g)
    ids[M // 3:M // 3 + 150] = -1
    p = problem(M, N, K, R, L, "bf16", rows, ids)
    got = lr().lora_add(**p)
    check(got, p, "bf16")
    base = p["base"].clone()
    assert torch.equal(lr().lora_add(**{**p, "base": base}, out=base), got)
