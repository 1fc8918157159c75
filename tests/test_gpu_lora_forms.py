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
