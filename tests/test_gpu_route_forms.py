"""GPU tests of the router and the sum of rows (include/route.h): forms that their kernels
take for certain sizes, types and masks, and what must hold between them."""
import pytest

from gpu_helpers import lib, say
from test_gpu_route import check_routing, define, define_backward, make_logits

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


# ---- sizes from which the kernels go on in another way

@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,E,top", [(40000, 60, 6), (20000, 256, 8), (70000, 130, 3),
                                     (5000, 1000, 8)])
def test_route_backward_of_several_tokens_a_group(T, E, top, dtype):
    """More tokens than groups of lanes are there at once: each takes several in turn, with what
    the weights pull at in the same memory and the loss's slopes kept.  Bar: as in
    test_gpu_route.py."""
    say(f"route backward T={T} E={E} top={top} {dtype}")
    logits = make_logits(T, E, dtype, T)
    g = torch.Generator().manual_seed(E)
    valid, a = torch.rand(T, generator=g) > 0.2, torch.randn(T, top, generator=g)
    for renormalize in (True, False):
        want = define(logits, top, renormalize, valid)
        r = rt().route_tokens(logits.cuda(), top, renormalize=renormalize, balance=True,
                              valid=valid.cuda())
        check_routing(r, want, True)
        got = rt().route_tokens_backward(logits.cuda(), r, a.cuda(),
                                         torch.tensor(40.0, device="cuda"))
        d, m = define_backward(want, a.double(), 40.0, renormalize)
        bound = (4 * min(want["D"], 104.0) + 160) * U * m + HALF[dtype] * d.abs() + TINY[dtype]
        assert bool(((got.cpu().double() - d).abs() <= bound).all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,top,N", [(2049, 2, 1031), (3000, 5, 4099), (2048, 2, 4099),
                                     (4000, 9, 72)])
def test_combine_backward_of_many_tokens(T, top, N, dtype):
    """Workgroups of 256 up to 2048 tokens, of 512 above.  Bar: as in test_gpu_route.py."""
    say(f"combine backward T={T} top={top} N={N} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    y = torch.randn(T * top, N, generator=g, device="cuda").to(DT[dtype])
    dout = torch.randn(T, N, generator=g, device="cuda").to(DT[dtype])
    w = torch.randn(T, top, generator=g, device="cuda")
    slots = torch.arange(T * top, device="cuda")
    lost = torch.rand(T * top, generator=g, device="cuda") < 0.1
    routed = int((~lost).sum())
    there = slots[~lost][torch.randperm(routed, generator=g, device="cuda")]
    places = torch.full((T * top,), -1, dtype=torch.int32, device="cuda")
    places[there] = torch.arange(routed, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, routed], dtype=torch.int32, device="cuda")
    dy, dw = rt().combine_rows_backward(dout, y, w, places.view(T, top), off)
    steps = 8 * -(-N // 2048) + 10
    # tokens' slots in the order of y's rows, a few thousand at a time
    assert bool((dw.reshape(-1)[lost] == 0).all()) and bool((dy[routed:] == 0).all())
    for first in range(0, routed, 4096):
        at = there[first:first + 4096]
        d, x = dout[at // top].double(), y[first:first + at.numel()].double()
        prod, scale = d * x, w.reshape(-1)[at].double()[:, None]
        assert bool(((dw.reshape(-1)[at].double() - prod.sum(1)).abs()
                     <= steps * U * prod.abs().sum(1) + 2.0 ** -126).all())
        want = d * scale
        assert bool(((dy[first:first + at.numel()].double() - want).abs()
                     <= (HALF[dtype] * (1 + U) + U) * want.abs() + TINY[dtype]).all())


@pytest.mark.parametrize("N", [8, 5, 2056])
def test_combine_of_more_tokens_than_one_launch_takes(N):
    """A launch takes 2^22 workgroups: 2^22 tokens, half as many of more than 2048 columns.
    Whole numbers, so that every step is exact."""
    T = (1 << 22) + 5 if N < 100 else (1 << 21) + 5
    say(f"combine of {T} tokens of {N}")
    t = torch.arange(T, device="cuda")
    n = torch.arange(N, device="cuda")
    y = (((t % 61).to(torch.int16)[:, None] + (n % 61).to(torch.int16)) % 61).to(torch.bfloat16)
    places = (T - 1 - t).to(torch.int32)[:, None].contiguous()
    w = (t % 3).float()[:, None]
    out = rt().combine_rows(y, w, places)
    assert torch.equal(out, y.flip(0) * w.to(torch.bfloat16))
    if N > 100:
        return
    off = torch.tensor([T - 2], dtype=torch.int32, device="cuda")
    dy, dw = rt().combine_rows_backward(y, y, w, places, off)
    want = (y * w.to(torch.bfloat16)).flip(0)          # row T - 1 - t is w[t] y[t]
    want[T - 2:] = 0
    assert torch.equal(dy, want)
    dots = (y.float() * y.flip(0).float()).sum(1)
    dots[:2] = 0                                       # places T - 1 and T - 2
    assert torch.equal(dw[:, 0], dots)
