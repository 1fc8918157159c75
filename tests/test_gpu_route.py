"""GPU tests of the router and the experts' sum (include/route.h) against their definitions
in 64 bits.

Bars, derived from the roundings counted below (u = 2^-24, half a step of fp32):
  * what is chosen, counts and the order are whole numbers and equal.
  * p: the difference to the row's maximum is off by u |l - max| at most, the exponential by
    4 u, the sum (16 in a lane, 6 steps over lanes) by 22 u, reciprocal and product by 3 u:
    P(D) = (D + 32) u, D the row's spread over what is not -infinity.  A renormalised weight
    replaces one sum by another of at most 32: (2 D + 48) u.
  * loss: sums of p over a tile, its waves, runs of tiles and experts: at most 64 + 16 + 16 +
    64 + 16 + 16 + 6 + 16 additions, two roundings in pull: (D + 300) u.
  * dlogits: p, weights, two sums of at most 22 terms and 6 more roundings, relative to the sum of
    the magnitudes that are added, then half a step of the output's type.
  * sums of rows: top + 1 fused steps, then half a step of the type; inner products: 8
    ceil(N / 2048) steps in a lane, 6 + 4 joined.
"""
import pytest

from gpu_helpers import lib, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    lib()


def rt():
    from w4a16_dequant_gemm_amd import route
    return route


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half a step of the smallest numbers, which fp32 flushes as a whole."""
    f = torch.finfo(dtype)
    return f.smallest_normal * (1.0 if dtype == torch.float32 else f.eps / 2)


def define(logits, top, renormalize, valid):
    """The definition, on the CPU in 64 bits."""
    l = logits.detach().cpu().double()
    T, E = l.shape
    ok = torch.ones(T, dtype=torch.bool) if valid is None else valid.cpu() != 0
    high = l.amax(1, keepdim=True) if E else l
    e = torch.where(high == -INF, 0.0, torch.exp(l - torch.where(high == -INF, 0.0, high)))
    total = e.sum(1, keepdim=True)
    p = torch.where(total == 0, 0.0, e / torch.where(total == 0, 1.0, total))
    p = torch.where(ok[:, None], p, 0.0)
    rank = torch.where(l == l, l, -INF)
    order = torch.sort(rank, dim=1, descending=True, stable=True)
    chosen, value = order.indices[:, :top], order.values[:, :top]
    there = (value > -INF) & ok[:, None]
    w = torch.where(there, p.gather(1, chosen), 0.0)
    if renormalize:
        s = w.sum(1, keepdim=True)
        w = torch.where(s == 0, 0.0, w / torch.where(s == 0, 1.0, s))
        w = torch.where(there, w, 0.0)
    experts = torch.where(there, chosen, -1)
    counts = torch.bincount(experts[there], minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64)
    offsets[1:] = counts.cumsum(0)
    flat = torch.where(there, chosen, E).reshape(-1)
    by = torch.argsort(flat, stable=True)
    n = int(offsets[-1])
    rows = torch.full((T * top,), -1, dtype=torch.int64)
    rows[:n] = by[:n] // top
    places = torch.full((T * top,), -1, dtype=torch.int64)
    places[by[:n]] = torch.arange(n)
    V = int(ok.sum())
    pull = counts.double() * (E / (V * top) / V if V else 0.0)
    loss = (pull * p.sum(0)).sum() if V else torch.zeros((), dtype=torch.float64)
    spread = torch.where(l > -INF, high - l, 0.0).amax(1)
    return dict(p=p, weights=w, experts=experts, counts=counts, offsets=offsets, rows=rows,
                places=places.view(T, top), pull=pull, loss=loss, V=V,
                D=float(spread.max()) if T else 0.0)


WHOLE = ("experts", "counts", "offsets", "rows", "places")


def check_routing(r, want, balance, what=""):
    for k in WHOLE:
        assert torch.equal(getattr(r, k).cpu().long(), want[k]), f"{what}: {k}"
    D = min(want["D"], 104.0)
    off = (r.weights.cpu().double() - want["weights"]).abs()
    assert bool((off <= (2 * D + 48) * U * want["weights"] + 2.0 ** -120).all()), what
    if balance:
        assert bool(((r.pull.cpu().double() - want["pull"]).abs() <= 2 * U * want["pull"]).all())
        assert abs(float(r.loss) - float(want["loss"])) <= (D + 300) * U * float(want["loss"]), what
    else:
        assert r.loss is None and r.pull is None


def make_logits(T, E, dtype, seed, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * scale).to(DT[dtype])


# E: each number of elements a lane can hold and its neighbours, both widths of groups;
# T: one workgroup, its limit, tiles of every size with a rest
SHAPES = [(1, 1, 1), (1, 64, 8), (3, 5, 5), (16, 16, 1), (17, 17, 2), (63, 64, 8), (64, 128, 32),
          (65, 60, 6), (64, 1024, 8), (100, 33, 4), (130, 256, 8), (257, 255, 3), (200, 257, 8),
          (515, 512, 8), (300, 1000, 32), (129, 1024, 1), (2049, 8, 2), (1040, 65, 4)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,E,top", SHAPES)
def test_route(T, E, top, dtype):
    say(f"route T={T} E={E} top={top} {dtype}")
    logits = make_logits(T, E, dtype, T + E)
    g = torch.Generator().manual_seed(E)
    padded = torch.rand(T, generator=g) > 0.3
    for renormalize, balance, valid in ((True, False, None), (False, True, None),
                                        (True, True, padded), (False, False, padded)):
        want = define(logits, top, renormalize, valid)
        r = rt().route_tokens(logits.cuda(), top, renormalize=renormalize, balance=balance,
                              valid=None if valid is None else valid.cuda())
        torch.cuda.synchronize()
        check_routing(r, want, balance, f"{renormalize} {balance} {valid is not None}")


@pytest.mark.parametrize("T", [16383, 16385, 32769, 70001])
def test_route_many_tokens(T):
    """Tiles of 16, 32 and 64 tokens, more tiles than one pass over them adds up."""
    say(f"route T={T}")
    logits = make_logits(T, 40, "bf16", T)
    want = define(logits, 4, True, None)
    r = rt().route_tokens(logits.cuda(), 4, balance=True)
    torch.cuda.synchronize()
    check_routing(r, want, True)


@pytest.mark.parametrize("T", [0, 5, 100])
def test_no_token_is_real(T):
    say(f"route without a real token, T={T}")
    logits = make_logits(T, 12, "fp32", 1).cuda()
    valid = torch.zeros(T, dtype=torch.uint8, device="cuda")
    r = rt().route_tokens(logits, 3, balance=True, valid=valid)
    assert torch.equal(r.counts.cpu(), torch.zeros(12, dtype=torch.int32))
    assert torch.equal(r.offsets.cpu(), torch.zeros(13, dtype=torch.int32))
    assert float(r.loss) == 0.0 and bool((r.pull == 0).all())
    assert bool((r.rows == -1).all()) and bool((r.experts == -1).all())
    assert bool((r.places == -1).all()) and bool((r.weights == 0).all())
    d = rt().route_tokens_backward(logits, r, torch.ones(T, 3, device="cuda"),
                                   torch.ones((), device="cuda"))
    assert d.shape == (T, 12) and bool((d == 0).all())


@pytest.mark.parametrize("T", [40, 300])
def test_equal_logits_go_to_the_lowest_index(T):
    """A few distinct values, so that lanes and neighbours within a lane tie; zeros of both
    signs are equal."""
    g = torch.Generator().manual_seed(7)
    for E in (16, 100, 256, 700):
        say(f"ties T={T} E={E}")
        logits = torch.randint(-1, 2, (T, E), generator=g).float()
        logits[::2] *= -1.0          # negative zeros
        logits[1] = 0.5              # a row of one value
        for dtype in ("fp32", "bf16"):
            want = define(logits, 8, True, None)
            r = rt().route_tokens(logits.to(DT[dtype]).cuda(), 8)
            torch.cuda.synchronize()
            check_routing(r, want, False)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,E", [(50, 20), (300, 20), (300, 300)])
def test_masked_experts(T, E, dtype):
    """-infinity and the type's lowest value: the first is never chosen, the second is when
    nothing else is left."""
    say(f"masked experts T={T} E={E} {dtype}")
    logits = make_logits(T, E, dtype, 3)
    logits[:, 5] = -INF
    logits[::3, 2:] = -INF           # two are left for six slots
    logits[1::3, 3:] = torch.finfo(DT[dtype]).min
    logits[4] = -INF
    logits[7] = torch.finfo(DT[dtype]).min
    for renormalize in (True, False):
        want = define(logits, 6, renormalize, None)
        want["D"] = 104.0            # what lies below is 0 in both
        r = rt().route_tokens(logits.cuda(), 6, renormalize=renormalize, balance=True)
        torch.cuda.synchronize()
        check_routing(r, want, True)
        d = rt().route_tokens_backward(logits.cuda(), r, torch.ones(T, 6, device="cuda"),
                                       torch.ones((), device="cuda"))
        assert bool(torch.isfinite(d).all())
        # row 7 holds the lowest value in column 5 too: 1/E of its probability
        assert bool((d.cpu()[logits == -INF] == 0).all())


@pytest.mark.parametrize("bad", [float("nan"), INF])
@pytest.mark.parametrize("T", [40, 300])
def test_what_is_not_finite_stays_in_its_row(bad, T):
    say(f"{bad} in one row, T={T}")
    logits = make_logits(T, 50, "fp32", 9)
    clean = rt().route_tokens(logits.cuda(), 4, balance=True)
    spoiled = logits.clone()
    spoiled[17, 3] = bad
    for renormalize in (True, False):
        clean = rt().route_tokens(logits.cuda(), 4, renormalize=renormalize)
        r = rt().route_tokens(spoiled.cuda(), 4, renormalize=renormalize, balance=True)
        others = torch.arange(T) != 17
        assert torch.equal(r.weights.cpu()[others], clean.weights.cpu()[others])
        assert bool(torch.isnan(r.weights[17]).any()) and bool(torch.isnan(r.loss))
        want = define(torch.where(spoiled == spoiled, spoiled, -INF), 4, renormalize, None)
        for k in WHOLE:
            assert torch.equal(getattr(r, k).cpu().long(), want[k]), k
        d = rt().route_tokens_backward(spoiled.cuda(), r, torch.ones(T, 4, device="cuda"))
        assert bool(torch.isnan(d[17]).any()) and bool(torch.isfinite(d[others.cuda()]).all())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_strided_and_unaligned_logits(dtype):
    big = make_logits(200, 150, dtype, 21).cuda()
    for first, E in ((0, 64), (1, 64), (3, 61), (8, 128), (6, 96)):
        say(f"columns {first}..{first + E} {dtype}")
        part = big[:, first:first + E]
        want = define(part, 5, True, None)
        r = rt().route_tokens(part, 5, balance=True)
        check_routing(r, want, True)
        alone = rt().route_tokens(part.contiguous(), 5, balance=True)
        for k in WHOLE + ("weights", "loss"):
            assert torch.equal(getattr(r, k), getattr(alone, k))
        dw = torch.rand(200, 5, device="cuda")
        assert torch.equal(rt().route_tokens_backward(part, r, dw, r.loss),
                           rt().route_tokens_backward(part.contiguous(), r, dw, r.loss))


def test_offsets_beyond_32_bits():
    """Logits of more than 4 GiB: the last rows are their own."""
    T, E = (1 << 21) + 70, 1024
    say(f"route T={T} E={E}")
    logits = torch.zeros(T, E, dtype=torch.float16, device="cuda")
    logits[:, 9] = 4.0
    tail = make_logits(70, E, "fp16", 2)
    logits[-70:] = tail.cuda()
    r = rt().route_tokens(logits, 1, renormalize=False)
    want = define(tail, 1, False, None)
    assert torch.equal(r.experts[-70:].cpu().long(), want["experts"])
    assert int(r.counts[9]) == T - 70 + int(want["counts"][9])
    assert bool((r.experts[:-70] == 9).all())
    assert torch.equal(r.rows[r.places.view(-1).long()], torch.arange(T, dtype=torch.int32,
                                                                      device="cuda"))
    d = rt().route_tokens_backward(logits, r, torch.ones(T, 1, device="cuda"))
    small = rt().route_tokens(tail.cuda(), 1, renormalize=False)
    assert torch.equal(d[-70:], rt().route_tokens_backward(tail.cuda(), small,
                                                           torch.ones(70, 1, device="cuda")))


# ---- the router's gradient

def define_backward(want, a, g, renormalize):
    """(dlogits, the sum of the magnitudes that are added) of a routing `want`."""
    p, w, pull = want["p"], want["weights"], want["pull"]
    a = torch.where(want["experts"] >= 0, a, 0.0)
    mean = (p * pull).sum(1, keepdim=True)
    S = (a * w).sum(1, keepdim=True)
    size = (a * w).abs().sum(1, keepdim=True)
    d = g * p * (pull - mean)
    m = abs(g) * p * (pull.abs() + mean.abs())
    at = want["experts"].clamp(min=0)
    if renormalize:
        d.scatter_add_(1, at, w * (a - S))
        m.scatter_add_(1, at, w * (a.abs() + size))
    else:
        d.scatter_add_(1, at, w * a)
        m.scatter_add_(1, at, w * a.abs())
        d -= p * S
        m += p * size
    return d, m


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (1, 64, 8), (3, 5, 5), (17, 17, 2), (66, 60, 6),
                                     (130, 256, 8), (40, 257, 32), (33, 1000, 4), (100, 128, 16),
                                     (50, 31, 20)])
def test_route_backward(T, E, top, dtype):
    say(f"route backward T={T} E={E} top={top} {dtype}")
    logits = make_logits(T, E, dtype, T * E)
    gen = torch.Generator().manual_seed(T)
    padded = torch.rand(T, generator=gen) > 0.3
    a = torch.randn(T, top, generator=gen)
    for renormalize, valid, with_a, g in ((True, None, True, None), (False, None, True, None),
                                          (True, padded, True, 0.7), (False, padded, True, -0.7),
                                          (True, None, False, 1.3), (False, None, False, None)):
        want = define(logits, top, renormalize, valid)
        r = rt().route_tokens(logits.cuda(), top, renormalize=renormalize, balance=g is not None,
                              valid=None if valid is None else valid.cuda())
        got = rt().route_tokens_backward(
            logits.cuda(), r, a.cuda() if with_a else None,
            None if g is None else torch.tensor(g, device="cuda"))
        torch.cuda.synchronize()
        d, m = define_backward(want, a.double() if with_a else torch.zeros(T, top).double(),
                               0.0 if g is None else g, renormalize)
        assert got.dtype == DT[dtype] and got.shape == (T, E)
        bound = (4 * min(want["D"], 104.0) + 160) * U * m + half_step(DT[dtype]) * d.abs() \
            + tiny(DT[dtype])
        assert bool(((got.cpu().double() - d).abs() <= bound).all())


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward_against_differences(renormalize):
    """The definition's own differences in 64 bits: no logit comes near a tie."""
    say(f"route gradient against differences, renormalize={renormalize}")
    T, E, top, g, step = 5, 9, 3, 0.8, 1e-6
    gen = torch.Generator().manual_seed(4)
    logits = torch.stack([torch.randperm(E, generator=gen) for _ in range(T)]).float() * 0.4
    a = torch.randn(T, top, generator=gen).double()
    counts = define(logits, top, renormalize, None)["pull"]

    def value(l):
        w = define(l, top, renormalize, None)
        return (a * w["weights"]).sum() + g * (counts * w["p"].sum(0)).sum()
    want = torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        for e in range(E):
            l = logits.double().clone()
            l[t, e] += step
            up = value(l)
            l[t, e] -= 2 * step
            want[t, e] = (up - value(l)) / (2 * step)
    r = rt().route_tokens(logits.cuda(), top, renormalize=renormalize, balance=True)
    got = rt().route_tokens_backward(logits.cuda(), r, a.float().cuda(),
                                     torch.tensor(g, device="cuda"))
    # fp32: 2^-24 of terms below 4; differences: step^2 and 2^-52 * 8 / step
    assert bool(((got.cpu().double() - want).abs() <= 200 * U * 4 + 1e-8).all())


# ---- the experts' sum

def make_rows(T, top, N, dtype, seed, lost=0.2, extra_rows=0):
    g = torch.Generator().manual_seed(seed)
    R = T * top + extra_rows
    places = torch.randperm(R, generator=g)[:T * top].view(T, top)
    places[torch.rand(T, top, generator=g) < lost] = -1
    return (torch.randn(R, N, generator=g).to(DT[dtype]), torch.randn(T, top, generator=g),
            places.to(torch.int32), torch.randn(T, N, generator=g).to(DT[dtype]))


ROWS = [(1, 1, 1), (1, 8, 4096), (3, 2, 7), (5, 3, 2831), (2, 4, 2048), (7, 5, 2056), (4, 8, 4099),
        (9, 11, 264), (2, 32, 40), (300, 6, 129), (1, 2, 20000)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,top,N", ROWS)
def test_combine(T, top, N, dtype):
    say(f"combine T={T} top={top} N={N} {dtype}")
    y, w, places, residual = make_rows(T, top, N, dtype, T + N)
    there = (places >= 0)[..., None]
    terms = torch.where(there, w.double()[..., None] * y.double()[places.clamp(min=0).long()], 0.0)
    for with_r in (True, False):
        want = terms.sum(1) + (residual.double() if with_r else 0.0)
        size = terms.abs().sum(1) + (residual.double().abs() if with_r else 0.0)
        got = rt().combine_rows(y.cuda(), w.cuda(), places.cuda(),
                                residual=residual.cuda() if with_r else None)
        torch.cuda.synchronize()
        bound = (top + 1) * U * size + half_step(DT[dtype]) * (want.abs() + top * U * size) \
            + tiny(DT[dtype])
        assert bool(((got.cpu().double() - want).abs() <= bound).all())
        if with_r:      # in place
            again = residual.cuda()
            assert rt().combine_rows(y.cuda(), w.cuda(), places.cuda(), residual=again,
                                     out=again) is again
            assert torch.equal(again, got)


def test_combine_leaves_unnamed_rows_unread():
    """Rows without a slot, weights of slots without a row, and places out of range."""
    y, w, places, _ = make_rows(6, 4, 100, "bf16", 3, lost=0.0, extra_rows=5)
    places[0, 1], places[1, 0], places[2, 3] = -5, 29, 1 << 30
    named = torch.zeros(29, dtype=torch.bool)
    named[places[(places >= 0) & (places < 29)].long()] = True
    clean = y.clone()
    clean[~named] = 0
    y[~named] = float("nan")
    w_bad = w.clone()
    w_bad[0, 1] = w_bad[1, 0] = w_bad[2, 3] = float("nan")
    a = rt().combine_rows(y.cuda(), w_bad.cuda(), places.cuda())
    b = rt().combine_rows(clean.cuda(), w.cuda(), places.cuda())
    assert bool(torch.isfinite(a).all()) and torch.equal(a, b)
    empty = rt().combine_rows(y[:0].cuda(), w.cuda(), places.cuda())
    assert bool((empty == 0).all())
    none = rt().combine_rows(y.cuda(), w[:0].cuda(), places[:0].cuda())
    assert none.shape == (0, 100)


@pytest.mark.parametrize("first,N", [(0, 96), (1, 97), (4, 64), (7, 1)])
def test_combine_strided(first, N):
    say(f"combine of columns {first}..{first + N}")
    y, w, places, residual = make_rows(9, 3, 120, "fp16", 8, lost=0.0)
    yd, rd, wd, pd = y.cuda(), residual.cuda(), w.cuda(), places.cuda()
    got = rt().combine_rows(yd[:, first:first + N], wd, pd, residual=rd[:, first:first + N])
    want = rt().combine_rows(yd, wd, pd, residual=rd)[:, first:first + N]
    assert torch.equal(got, want)
    off = torch.tensor([0, 27], dtype=torch.int32, device="cuda")    # every row has its slot
    a = rt().combine_rows_backward(rd[:, first:first + N], yd[:, first:first + N], wd, pd, off)
    b = rt().combine_rows_backward(rd[:, first:first + N].contiguous(),
                                   yd[:, first:first + N].contiguous(), wd, pd, off)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,top,N", ROWS)
def test_combine_backward(T, top, N, dtype):
    say(f"combine backward T={T} top={top} N={N} {dtype}")
    y, w, _, dout = make_rows(T, top, N, dtype, T * N)
    logits = make_logits(T, max(top, 7), "fp32", N)
    valid = torch.arange(T) % 3 != 1
    r = define(logits, top, True, valid)
    places, n = r["places"].to(torch.int32), int(r["offsets"][-1])
    dy, dw = rt().combine_rows_backward(dout.cuda(), y.cuda(), w.cuda(), places.cuda(),
                                        r["offsets"].to(torch.int32).cuda())
    torch.cuda.synchronize()
    there = (places >= 0)[..., None]
    at = places.clamp(min=0).long()
    prod = torch.where(there, dout.double()[:, None] * y.double()[at], 0.0)
    steps = 8 * -(-N // 2048) + 10
    bound = steps * U * prod.abs().sum(-1) + 2.0 ** -126
    assert bool(((dw.cpu().double() - prod.sum(-1)).abs() <= bound).all())
    want = torch.zeros(T * top, N, dtype=torch.float64)
    want[at[there[..., 0]]] = (w.double()[..., None] * dout.double()[:, None])[there[..., 0]]
    assert bool(((dy.cpu().double() - want).abs()
                 <= (half_step(DT[dtype]) * (1 + U) + U) * want.abs() + tiny(DT[dtype])).all())
    assert bool((dy[n:] == 0).all())


def test_rows_behind_the_last_stay_zeros():
    """A place at or behind the routed rows is none at all: nothing else writes there."""
    y, w, places, dout = (t.cuda() for t in make_rows(8, 2, 64, "bf16", 4, lost=0.0))
    off = torch.tensor([0, 11], dtype=torch.int32, device="cuda")
    dy, dw = rt().combine_rows_backward(dout, y, w, places, off)
    full, dw_full = rt().combine_rows_backward(dout, y, w, places, off + 5)
    assert bool((dy[11:] == 0).all()) and torch.equal(dy[:11], full[:11])
    assert torch.equal(dw, torch.where(places < 11, dw_full, 0.0))


def test_combine_backward_against_differences():
    """Both gradients of a linear map: its own differences, in 64 bits."""
    say("combine gradient against differences")
    y, w, places, c = make_rows(4, 3, 10, "bf16", 6, lost=0.0)

    def value(y, w):
        return (c.double() * (w[..., None] * y[places.long()]).sum(1)).sum()
    off = torch.tensor([0, 12], dtype=torch.int32)
    dy, dw = rt().combine_rows_backward(c.cuda(), y.cuda(), w.cuda(), places.cuda(), off.cuda())
    y, w = y.double(), w.double()
    for r, n in ((0, 0), (5, 9), (11, 4)):
        e = torch.zeros_like(y)
        e[r, n] = 1.0
        want = value(y + e, w) - value(y, w)
        assert abs(float(dy[r, n]) - float(want)) <= 2.0 ** -8 * abs(float(want)) + 1e-12
    for t, j in ((0, 0), (3, 2)):
        e = torch.zeros_like(w)
        e[t, j] = 1.0
        want = value(y, w + e) - value(y, w)
        assert abs(float(dw[t, j]) - float(want)) <= 1e-5


def test_combine_offsets_beyond_32_bits():
    T, top, N = 33000, 2, 40000
    say(f"combine of {T * top} rows of {N}")
    y = torch.zeros(T * top, N, dtype=torch.bfloat16, device="cuda")
    y[-1] = 3.0
    places = torch.arange(T * top, dtype=torch.int32, device="cuda").view(T, top)
    w = torch.full((T, top), 0.5, device="cuda")
    out = rt().combine_rows(y, w, places)
    assert bool((out[-1] == 1.5).all()) and bool((out[-2] == 0).all())
    off = torch.tensor([T * top - 1], dtype=torch.int32, device="cuda")
    places[-1, -1] = -1
    out.fill_(2.0)
    dy, dw = rt().combine_rows_backward(out, y, w, places, off)
    assert bool((dy[-2] == 1.0).all()) and bool((dy[-1] == 0).all()) and float(dw[-1, -1]) == 0.0


# ---- streams and graphs

def test_equal_calls_give_equal_bits():
    for T in (40, 700):
        logits = make_logits(T, 100, "fp32", 1).cuda()
        runs = [rt().route_tokens(logits, 8, balance=True) for _ in range(4)]
        for r in runs[1:]:
            for k in WHOLE + ("weights", "loss", "pull"):
                assert torch.equal(getattr(r, k), getattr(runs[0], k)), k


def test_on_another_stream():
    logits = make_logits(700, 64, "bf16", 5).cuda()
    want = rt().route_tokens(logits, 8, balance=True)
    y, w, places, res = (t.cuda() for t in make_rows(700, 8, 256, "bf16", 5))
    sums = rt().combine_rows(y, w, places, residual=res)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    big = torch.rand(4096, 4096, device="cuda")
    for _ in range(20):
        big = big @ big * 1e-3      # the current stream is at work
    r = rt().route_tokens(logits, 8, balance=True, stream=side)
    d = rt().route_tokens_backward(logits, r, w, r.loss, stream=side)
    c = rt().combine_rows(y, w, places, residual=res, stream=side)
    side.synchronize()
    for k in WHOLE + ("weights", "loss"):
        assert torch.equal(getattr(r, k).cpu(), getattr(want, k).cpu())
    assert torch.equal(c.cpu(), sums.cpu())
    torch.cuda.synchronize()
    assert torch.equal(d, rt().route_tokens_backward(logits, want, w, want.loss))


@pytest.mark.parametrize("T", [20, 700])
def test_graph_replays_match_eager(T):
    """Two graphs of different sizes, replayed in turn with eager calls between."""
    say(f"graphs T={T}")
    made = []
    for n, seed in ((T, 1), (T + 300, 2)):
        logits = make_logits(n, 64, "bf16", seed).cuda()
        dw = torch.randn(n, 8, device="cuda")
        y = torch.randn(n * 8, 200, device="cuda").to(torch.bfloat16)

        def step(logits=logits, dw=dw, y=y):
            r = rt().route_tokens(logits, 8, balance=True)
            d = rt().route_tokens_backward(logits, r, dw, r.loss)
            out = rt().combine_rows(y, r.weights, r.places)
            dy, dcw = rt().combine_rows_backward(out, y, r.weights, r.places, r.offsets)
            return [r.weights, r.experts, r.rows, r.places, r.offsets, r.loss, d, out, dy, dcw]
        eager = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        made.append((graph, outs, eager, step))
    for rep in range(3):
        for graph, outs, _, _ in made:
            for t in outs:
                t.zero_()
        for graph, *_ in reversed(made):
            graph.replay()
        made[0][3]()
        torch.cuda.synchronize()
        for _, outs, eager, _ in made:
            assert all(torch.equal(a, b) for a, b in zip(outs, eager)), rep


# ---- together with the products

def test_a_block_of_experts():
    """Router, grouped products, gated activation and sum: as the example runs them, against
    the same products in an order made by torch."""
    from w4a16_dequant_gemm_amd import fp8, rowquant
    say("a block of experts")
    T, E, top, H, F = 133, 10, 3, 256, 384
    g = torch.Generator().manual_seed(12)
    x, res = (torch.randn(T, H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    logits = torch.randn(T, E, generator=g)
    valid = torch.arange(T) < 120
    E4M3 = torch.float8_e4m3fn
    up = fp8.fp8_repack((torch.randn(E, 2 * F, H, generator=g) * 30).to(E4M3).cuda(),
                        torch.full((E, 6, 2), 2e-3).cuda())
    down = fp8.fp8_repack((torch.randn(E, H, F, generator=g) * 30).to(E4M3).cuda(),
                          torch.full((E, 2, 3), 2e-3).cuda())
    q, s, h = rowquant.rmsnorm_quantize_rows(x, torch.ones(H, dtype=torch.bfloat16).cuda(),
                                             residual=res)

    def experts(offsets, rows):
        both = fp8.fp8_grouped_gemm(q, s, up, offsets, rows=rows)
        return fp8.fp8_grouped_gemm(*rowquant.swiglu_quantize_rows(both[:, :F], both[:, F:]), down,
                                    offsets)
    r = rt().route_tokens(logits.cuda(), top, valid=valid.cuda())
    y = experts(r.offsets, r.rows)
    got = rt().combine_rows(y, r.weights, r.places, residual=h).cpu()

    want = define(logits, top, True, valid)
    n = int(want["offsets"][-1])
    y2 = experts(want["offsets"].to(torch.int32).cuda(), want["rows"].to(torch.int32).cuda())
    assert torch.equal(y[:n], y2[:n])
    back = y2.double().cpu()[want["places"].clamp(min=0)]
    terms = torch.where((want["places"] >= 0)[..., None], want["weights"][..., None] * back, 0.0)
    total = terms.sum(1) + h.double().cpu()
    size = terms.abs().sum(1) + h.double().cpu().abs()
    slack = (top + 1 + 2 * want["D"] + 48) * U * size
    assert bool(((got.double() - total).abs() <= slack * (1 + 2.0 ** -8) + 2.0 ** -8 * total.abs()
                 + 2.0 ** -133).all())
    assert torch.equal(got[120:], h.cpu()[120:])
