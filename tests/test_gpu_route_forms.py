"""GPU tests of the router and the sum of rows (include/route.h): forms that their kernels
take for certain sizes, types and masks, and what must hold between them."""
import pytest

from gpu_helpers import lib, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24                                      # half a step of fp32
HALF = {k: torch.finfo(v).eps / 2 for k, v in DT.items()}
# half a step of the smallest numbers (fp32: those it flushes)
TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134, "fp32": 2.0 ** -126}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    lib()


def rt():
    from w4a16_dequant_gemm_amd import route
    return route


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("top", [1, 2, 3, 4, 5, 6, 7, 8, 9, 17, 32])
def test_sum_of_rows_with_all_some_and_no_slots(top, dtype):
    """Every number of slots.  top fused steps of fp32, then half a step of the type; a token
    without a slot keeps its residual's bits (a -0 too), whatever its weights."""
    say(f"sum of rows, top={top} {dtype}")
    T, N = 40, 72
    g = torch.Generator().manual_seed(top)
    y = torch.randn(T * top, N, generator=g).to(DT[dtype])
    w = torch.randn(T, top, generator=g)
    res = torch.randn(T, N, generator=g).to(DT[dtype])
    res[:, ::3] = -0.0
    places = torch.randperm(T * top, generator=g).view(T, top).to(torch.int32)
    lost = torch.rand(T, top, generator=g) < torch.arange(T)[:, None] / (T - 4)
    lost[T - 4:] = True
    places[lost] = -1
    w[lost] = torch.where(torch.rand(T, top, generator=g) < 0.5, float("nan"), float("inf"))[lost]
    got = rt().combine_rows(y.cuda(), w.cuda(), places.cuda(), residual=res.cuda()).cpu()
    terms = torch.where(lost[..., None], 0.0,
                        w.double()[..., None] * y[places.clamp(min=0).long()].double())
    want = res.double() + terms.sum(1)
    size = res.double().abs() + terms.abs().sum(1)
    bound = top * U * size + HALF[dtype] * (want.abs() + top * U * size) + TINY[dtype]
    assert bool(((got.double() - want).abs() <= bound).all())
    none = lost.all(1)
    assert int(none.sum()) >= 4
    assert torch.equal(got[none].view(torch.int16), res[none].view(torch.int16))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("E,top", [(256, 8), (100, 6), (60, 3), (16, 8), (300, 8), (100, 11)])
@pytest.mark.parametrize("T", [64, 300])
def test_weights_do_not_depend_on_the_tokens_beside(T, E, top, dtype):
    """Tokens share a wave by fours; one with few logits that can be chosen, or with equal ones,
    sends all of them another way.  The others' outputs keep their bits."""
    say(f"weights beside other tokens T={T} E={E} top={top} {dtype}")
    g = torch.Generator().manual_seed(E + top)
    logits = (torch.randn(T, E, generator=g) * 2).to(DT[dtype])
    want = rt().route_tokens(logits.cuda(), top)
    at = torch.arange(T)
    for what in ("few", "nan", "equal"):
        bad = logits.clone()
        if what == "few":
            bad[3::4, 2:] = float("-inf")
        elif what == "nan":
            bad[3::4, 1:] = float("nan")
        else:
            bad[3::4] = 0.5
        got = rt().route_tokens(bad.cuda(), top)
        keep = at % 4 != 3
        assert torch.equal(got.experts.cpu()[keep], want.experts.cpu()[keep]), what
        assert torch.equal(got.weights.cpu()[keep].view(torch.int32),
                           want.weights.cpu()[keep].view(torch.int32)), what
