"""GPU tests of the block-scaled fp8 product, alone and grouped by expert (include/fp8.h),
against the definition in 64 bits.

Bar: |Y - y| <= (eps/2 |y| + tiny) for the one rounding to the output type + C B, with
y the definition's sum and B = sum of |terms|.  The matrix unit adds fp8 products in groups
of 8, aligned to the group's largest and kept to 13 binary places below it (measured with
single products), so a group is off by less than 8 * 2^-13 of its largest product.  The rest
are fp32 additions: 16 groups to a block, one fused multiply-add per block and one rounding
of the scales' product.  C = 2^-10 + (K/128 + 136) 2^-23.  Where all products of a sum are
small whole numbers and the scales powers of two nothing is lost, and outputs are equal bit
for bit: test_whole_numbers_are_exact.
"""
import pytest

from gpu_helpers import lib, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
E4M3 = torch.float8_e4m3fn
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
PLANS = [None, ("stream", 1), ("stream", 2), ("tiled", 1), ("tiled", 2), ("tiled", 3), ("tiled", 4),
         ("tiled", 5), ("tiled", 6)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    lib()


def f8():
    from w4a16_dequant_gemm_amd import fp8
    return fp8


def blocks(n):
    return -(-n // 128)


def make(T, K, N, E=None, seed=0):
    """Codes over the whole range of E4M3 without NaN, and uneven positive scales."""
    g = torch.Generator().manual_seed(seed)

    def codes(*shape):
        c = torch.randint(0, 127, shape, generator=g, dtype=torch.uint8)
        return c | (torch.randint(0, 2, shape, generator=g, dtype=torch.uint8) << 7)
    lead = () if E is None else (E,)
    xq, w = codes(T, K), codes(*lead, N, K)
    xs = torch.rand(T, blocks(K), generator=g) * 2e-3 + 1e-4
    ws = torch.rand(*lead, blocks(N), blocks(K), generator=g) * 2e-4 + 1e-5
    return xq.cuda().view(E4M3), xs.cuda(), w.cuda().view(E4M3), ws.cuda()


def values(q, s, per_row):
    N, K = q.shape
    s = s.double().repeat_interleave(128, 1)[:, :K]
    if not per_row:
        s = s.repeat_interleave(128, 0)[:N]
    return q.float().double() * s


def product(x, w):
    return x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()


def assert_close(Y, y, B, K, what):
    eps = torch.finfo(Y.dtype).eps
    tiny = torch.finfo(Y.dtype).smallest_normal * eps
    bound = y.abs() * eps / 2 + tiny / 2 + (2.0 ** -10 + (K / 128 + 136) * 2.0 ** -23) * B
    err = (Y.double() - y).abs()
    assert bool((err <= bound).all()), (what, float((err / bound.clamp(min=1e-300)).max()))


@pytest.mark.parametrize("out", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N", [
    (1, 16, 1), (1, 128, 128), (2, 144, 130), (15, 1024, 64), (16, 272, 257), (17, 4096, 96),
    (33, 2048, 500), (65, 400, 1001), (129, 1168, 384), (200, 640, 255), (300, 2064, 700),
    (8, 8208, 512), (257, 128, 260)])
def test_product(out, M, K, N):
    xq, xs, w, ws = make(M, K, N, seed=M + K)
    packed = f8().fp8_repack(w, ws)
    y, B = product(values(xq, xs, True), values(w, ws, False))
    for plan in PLANS:
        say(f"fp8 product {out} M={M} K={K} N={N} plan={plan}")
        Y = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
        f8().fp8_gemm(xq, xs, packed, out=out, Y=Y, plan=plan)
        torch.cuda.synchronize()
        assert_close(Y, y, B, K, plan)


def make_exact(T, K, N, E=None, seed=0):
    """Codes of -2 .. 2 and scales 2^-3 .. 2^0: a block's sum is a whole number up to 512
    and the total, in steps of 2^-6, stays below 2^18 up to K = 65536."""
    g = torch.Generator().manual_seed(seed)
    lead = () if E is None else (E,)

    def codes(*shape):
        return torch.randint(-2, 3, shape, generator=g).float().to(E4M3).cuda()

    def scales(*shape):
        return torch.exp2(-torch.randint(0, 4, shape, generator=g).float()).cuda()
    return (codes(T, K), scales(T, blocks(K)), codes(*lead, N, K),
            scales(*lead, blocks(N), blocks(K)))


@pytest.mark.parametrize("out", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K,N", [
    (1, 16, 3), (1, 8192, 640), (5, 1040, 130), (16, 4096, 128), (31, 1424, 77), (64, 8208, 256),
    (100, 7184, 513), (256, 1024, 256), (259, 2064, 1028), (520, 144, 136)])
def test_whole_numbers_are_exact(out, M, K, N):
    xq, xs, w, ws = make_exact(M, K, N, seed=M * 7 + K)
    packed = f8().fp8_repack(w, ws)
    want = product(values(xq, xs, True), values(w, ws, False))[0].to(DT[out])
    for plan in PLANS:
        say(f"fp8 exact {out} M={M} K={K} N={N} plan={plan}")
        Y = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
        f8().fp8_gemm(xq, xs, packed, out=out, Y=Y, plan=plan)
        torch.cuda.synchronize()
        assert torch.equal(Y, want), plan


@pytest.mark.parametrize("counts,K,N", [([3, 0, 17, 1], 272, 130), ([65, 300, 0, 2, 129], 1168, 520),
                                        ([9] * 40, 512, 96)])
def test_grouped_whole_numbers_are_exact(counts, K, N):
    E, R = len(counts), sum(counts)
    T = 2 * R // 3
    xq, xs, w, ws = make_exact(T, K, N, E=E, seed=K)
    packed = f8().fp8_repack(w, ws)
    idx = torch.randint(0, T, (R,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    x = values(xq, xs, True)[idx.long().cuda()]
    off = offsets_of(counts)
    ends = off.tolist()
    want = torch.cat([product(x[a:b], values(w[e], ws[e], False))[0]
                      for e, (a, b) in enumerate(zip(ends, ends[1:]))]).half()
    for plan in PLANS:
        say(f"fp8 grouped exact {counts[:5]} K={K} N={N} plan={plan}")
        Y = f8().fp8_grouped_gemm(xq, xs, packed, off, rows=idx.cuda(), out="fp16", plan=plan)
        torch.cuda.synchronize()
        assert torch.equal(Y, want), plan


def offsets_of(counts):
    off = torch.zeros(len(counts) + 1, dtype=torch.int32)
    off[1:] = torch.tensor(counts, dtype=torch.int32).cumsum(0)
    return off.cuda()


GROUPS = [
    ([0], 128, 128), ([3], 144, 130), ([0, 0, 5, 0], 256, 96), ([1, 16, 17, 0, 2], 400, 255),
    ([64, 0, 65, 63, 1, 0], 1024, 384), ([130, 257, 0, 1], 272, 520),
    ([1] * 70 + [0] * 60 + [3] * 70, 160, 64), ([600, 3], 2064, 256)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,K,N", GROUPS)
def test_grouped(counts, K, N, gather):
    E, R = len(counts), sum(counts)
    T = max(1, R // 3) if gather else R
    xq, xs, w, ws = make(T, K, N, E=E, seed=E + K)
    packed = f8().fp8_repack(w, ws)
    off = offsets_of(counts)
    g = torch.Generator().manual_seed(9)
    idx = torch.randint(0, T, (R,), generator=g, dtype=torch.int32).cuda() if gather else None
    x = values(xq, xs, True)
    if gather:
        x = x[idx.long()]
    y, B = torch.empty(R, N, dtype=torch.float64, device="cuda"), \
        torch.empty(R, N, dtype=torch.float64, device="cuda")
    at = 0
    for e, c in enumerate(counts):
        if c:
            y[at:at + c], B[at:at + c] = product(x[at:at + c], values(w[e], ws[e], False))
        at += c
    for plan in PLANS:
        say(f"fp8 grouped {counts[:6]} K={K} N={N} gather={gather} plan={plan}")
        Y = torch.full((R, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        f8().fp8_grouped_gemm(xq, xs, packed, off, rows=idx, out="bf16", Y=Y, plan=plan)
        torch.cuda.synchronize()
        assert_close(Y, y, B, K, plan)


def test_row_indices_outside_give_zeros():
    counts, K, N = [5, 0, 70], 272, 200
    xq, xs, w, ws = make(6, K, N, E=3, seed=4)
    packed = f8().fp8_repack(w, ws)
    idx = (torch.arange(75, dtype=torch.int32) % 6).cuda()
    bad = idx.clone()
    where = torch.tensor([0, 4, 5, 40, 74], device="cuda")
    bad[where] = torch.tensor([-1, 6, 2 ** 31 - 1, -2 ** 31, 1000], dtype=torch.int32,
                              device="cuda")
    off = offsets_of(counts)
    for plan in PLANS:
        say(f"row indices outside plan={plan}")
        want = f8().fp8_grouped_gemm(xq, xs, packed, off, rows=idx, plan=plan)
        got = f8().fp8_grouped_gemm(xq, xs, packed, off, rows=bad, plan=plan)
        want[where] = 0
        assert torch.equal(got, want)


def test_offsets_outside_are_taken_as_the_nearer_end():
    K, N = 256, 128
    xq, xs, w, ws = make(9, K, N, E=3, seed=5)
    packed = f8().fp8_repack(w, ws)
    good = torch.tensor([0, 4, 4, 9], dtype=torch.int32, device="cuda")
    wild = torch.tensor([-7, 4, 4, 1000], dtype=torch.int32, device="cuda")
    for plan in PLANS:
        say(f"offsets outside plan={plan}")
        want = f8().fp8_grouped_gemm(xq, xs, packed, good, plan=plan)
        got = f8().fp8_grouped_gemm(xq, xs, packed, wild, plan=plan)
        assert torch.equal(got, want)


def test_nan_codes_stay_in_their_row_and_column():
    M, K, N = 40, 400, 150
    xq, xs, w, ws = make(M, K, N, seed=6)
    for plan in PLANS:
        say(f"nan codes plan={plan}")
        want = f8().fp8_gemm(xq, xs, f8().fp8_repack(w, ws), plan=plan)
        x2, w2 = xq.clone(), w.clone()
        x2.view(torch.uint8)[17, 399] = 0x7F
        w2.view(torch.uint8)[149, 3] = 0xFF
        got = f8().fp8_gemm(x2, xs, f8().fp8_repack(w2, ws), plan=plan)
        nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
        nan[17] = True
        nan[:, 149] = True
        assert torch.equal(torch.isnan(got), nan)
        assert torch.equal(got[~nan], want[~nan])


def test_equal_calls_give_equal_bits():
    for M, K, N in ((5, 4096, 256), (100, 8192, 300), (300, 1024, 1000)):
        xq, xs, w, ws = make(M, K, N, seed=7)
        packed = f8().fp8_repack(w, ws)
        first = f8().fp8_gemm(xq, xs, packed)
        for _ in range(5):
            assert torch.equal(f8().fp8_gemm(xq, xs, packed), first)


def test_rows_do_not_depend_on_their_neighbours():
    """A row has the same bits in any batch that takes the same plan."""
    xq, xs, w, ws = make(64, 1024, 256, seed=8)
    packed = f8().fp8_repack(w, ws)
    for plan in PLANS[1:3]:
        whole = f8().fp8_gemm(xq, xs, packed, plan=plan)
        one = f8().fp8_gemm(xq[37:38].clone(), xs[37:38].clone(), packed, plan=plan)
        assert torch.equal(one[0], whole[37])


def test_no_rows():
    xq, xs, w, ws = make(1, 256, 128, E=2, seed=9)
    packed = f8().fp8_repack(w, ws)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert f8().fp8_grouped_gemm(xq, xs, packed, off, rows=none).shape == (0, 128)
    one = f8().fp8_repack(w[0].contiguous(), ws[0].contiguous())
    assert f8().fp8_gemm(xq[:0], xs[:0], one).shape == (0, 128)


def test_another_stream_and_a_graph():
    xq, xs, w, ws = make(100, 4096, 512, seed=10)
    packed = f8().fp8_repack(w, ws)
    exq, exs, ew, ews = make(60, 512, 256, E=4, seed=11)
    experts = f8().fp8_repack(ew, ews)
    off = offsets_of([10, 0, 49, 1])
    want = f8().fp8_gemm(xq, xs, packed), f8().fp8_grouped_gemm(exq, exs, experts, off)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = f8().fp8_gemm(xq, xs, packed), f8().fp8_grouped_gemm(exq, exs, experts, off)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = tuple(torch.empty_like(t) for t in want)
    ws_t = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f8().fp8_gemm(xq, xs, packed, Y=out[0], workspace=ws_t)
        f8().fp8_grouped_gemm(exq, exs, experts, off, Y=out[1])
    for rep in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), rep
        assert torch.equal(f8().fp8_gemm(xq, xs, packed, workspace=ws_t), want[0])


def test_refusals_on_the_device():
    from w4a16_dequant_gemm_amd import W4A16Error
    xq, xs, w, ws = make(4, 256, 128, E=2, seed=12)
    packed = f8().fp8_repack(w, ws)
    off = offsets_of([2, 2])
    for call in (lambda: f8().fp8_gemm(xq, xs, packed),
                 lambda: f8().fp8_repack(w, ws[:, :, :1].contiguous()),
                 lambda: f8().fp8_repack(w[:, :, :200], ws),
                 lambda: f8().fp8_grouped_gemm(xq, xs[:3], packed, off),
                 lambda: f8().fp8_grouped_gemm(xq[:, :128].contiguous(), xs, packed, off),
                 lambda: f8().fp8_grouped_gemm(xq, xs, packed, off[:2]),
                 lambda: f8().fp8_grouped_gemm(xq, xs, packed, off.long()),
                 lambda: f8().fp8_grouped_gemm(xq, xs, packed, off, rows=off.long())):
        with pytest.raises(W4A16Error):
            call()
    with pytest.raises(ValueError):
        f8().fp8_grouped_gemm(xq, xs, packed, off, out="i32")


def test_norm_product_activation_product():
    """The feed-forward path as a user runs it: each step against 64 bits from the rows
    the step before left."""
    from w4a16_dequant_gemm_amd import rowquant
    T, H, F = 37, 512, 640
    g = torch.Generator().manual_seed(13)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    r = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    wn = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    _, _, w1, s1 = make(1, H, 2 * F, seed=14)
    _, _, w2, s2 = make(1, F, H, seed=15)
    q, s, h = rowquant.rmsnorm_quantize_rows(x, wn, residual=r)
    both = f8().fp8_gemm(q, s, f8().fp8_repack(w1, s1))
    y, B = product(values(q, s, True), values(w1, s1, False))
    assert_close(both, y, B, H, "up")
    q2, sc2 = rowquant.swiglu_quantize_rows(both[:, :F], both[:, F:])
    out = f8().fp8_gemm(q2, sc2, f8().fp8_repack(w2, s2))
    y, B = product(values(q2, sc2, True), values(w2, s2, False))
    assert_close(out, y, B, F, "down")


def test_every_byte_of_a_blob_is_written():
    """Equal weights give equal blobs, whatever the memory held."""
    for E, K, N in ((None, 640, 130), (3, 144, 100), (None, 16, 1)):
        _, _, w, ws = make(1, K, N, E=E, seed=31)
        size = f8().fp8_packed_bytes(E or 1, K, N)
        say(f"blob bytes E={E} K={K} N={N}")
        blobs = []
        for fill in (0x00, 0xA5):
            data = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
            status = f8()._lib().fp8_repack(w.data_ptr(), ws.data_ptr(), E or 1, K, N,
                                            data.data_ptr(), size, None)
            torch.cuda.synchronize()
            assert status == 0
            blobs.append(data)
        assert torch.equal(*blobs)


def test_scales_from_any_place_in_a_tensor():
    """Rows and experts cut out of larger tensors: their scales start at any float."""
    K, N, E = 640, 130, 3                                # 5 scales a row, 10 an expert
    xq, xs, w, ws = make(70, K, N, E=E, seed=21)
    one = f8().fp8_repack(w[1].contiguous(), ws[1].clone())
    cut = f8().fp8_repack(w[1].contiguous(), ws[1])
    assert ws[1].data_ptr() % 16 and torch.equal(one.data, cut.data)
    experts = f8().fp8_repack(w, ws)
    off = offsets_of([20, 0, 47])
    for plan in PLANS:
        say(f"scales from any place plan={plan}")
        assert xs[3:].data_ptr() % 16
        want = f8().fp8_gemm(xq[3:].clone(), xs[3:].clone(), one, plan=plan)
        assert torch.equal(f8().fp8_gemm(xq[3:], xs[3:], one, plan=plan), want)
        want = f8().fp8_grouped_gemm(xq[3:].clone(), xs[3:].clone(), experts, off, plan=plan)
        assert torch.equal(f8().fp8_grouped_gemm(xq[3:], xs[3:], experts, off, plan=plan), want)


def plus_minus_one(*shape, seed):
    """Codes of 1 and -1, made in place (their number is large)."""
    x = torch.empty(shape, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = x.view(-1)
    for at in range(0, flat.numel(), 1 << 30):
        flat[at:at + (1 << 30)].random_(0, 2, generator=g).mul_(128).add_(0x38)
    return x.view(E4M3)


def test_more_tiles_than_one_launch_holds():
    """2^30 rows, the most there can be: 2^24 tiles of 64 rows and 256 threads are 2^32
    work-items, the rows 2^34 bytes."""
    M, K, N = 1 << 30, 16, 8
    xq, w = plus_minus_one(M, K, seed=41), plus_minus_one(2, N, K, seed=42)
    xs = torch.full((M, 1), 0.5, device="cuda")
    ws = torch.full((2, 1, 1), 0.5, device="cuda")
    blobs = [f8().fp8_repack(w[e], ws[e]) for e in range(2)]
    experts = f8().fp8_repack(w, ws)
    say(f"product of {M} rows")
    Y = f8().fp8_gemm(xq, xs, blobs[0])
    half = M // 2 + 17
    off = torch.tensor([0, half, M], dtype=torch.int32, device="cuda")
    places = [slice(at, at + 300) for at in (0, M // 8 - 150, half - 150, M - M // 8 - 150, M - 300)]
    for at in places:
        want = (xq[at].float().double() @ w[0].float().double().t().contiguous()) / 4
        assert torch.equal(Y[at].double(), want)
    say(f"grouped product of {M} rows")
    Y.fill_(float("nan"))
    f8().fp8_grouped_gemm(xq, xs, experts, off, Y=Y)
    for at in places:
        y = [xq[at].float().double() @ w[e].float().double().t().contiguous() / 4 for e in (0, 1)]
        own = torch.arange(at.start, at.stop, device="cuda")[:, None] >= half
        assert torch.equal(Y[at].double(), torch.where(own, y[1], y[0]))
    assert not bool(torch.isnan(Y.view(-1)[:1 << 31]).any())
    assert not bool(torch.isnan(Y.view(-1)[1 << 31:]).any())
    del xq, xs, Y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("plan", [("stream", 1), ("tiled", 3), None])
def test_the_most_experts(plan):
    """65535 experts of a row each but for some without: the streaming kernel's 136 strips
    each are more than one launch holds, and the blob has 2^34 bytes."""
    E, K, N = 65535, 16, 2176
    xq, w = plus_minus_one(E, K, seed=43), plus_minus_one(E, N, K, seed=44)
    xs = torch.full((E, 1), 0.5, device="cuda")
    ws = torch.full((E, 17, 1), 0.5, device="cuda")
    packed = f8().fp8_repack(w, ws)
    counts = torch.ones(E, dtype=torch.int64, device="cuda")
    counts[5::1000] = 0
    counts[7::1000] += 1
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = counts.cumsum(0)
    R = int(off[-1])
    rows = torch.randint(0, E, (R,), generator=torch.Generator().manual_seed(45)).to(torch.int32).cuda()
    say(f"{E} experts plan={plan}")
    Y = torch.full((R, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    f8().fp8_grouped_gemm(xq, xs, packed, off, rows=rows, Y=Y, plan=plan)
    torch.cuda.synchronize()
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), counts, output_size=R)
    for at in range(0, R, 8192):
        x = xq[rows[at:at + 8192].long()].float()
        want = (x[:, None, :] * w[expert[at:at + 8192]].float()).sum(-1) / 4
        assert torch.equal(Y[at:at + 8192].float(), want)
    del packed, w, Y
    torch.cuda.empty_cache()


# The 256 x 256 tile reads its scales four blocks at a time, the last group shifted back to
# end in the row: blocks of K by every remainder of four.
@pytest.mark.parametrize("K", [512, 640, 768, 896, 1104, 1248, 1392, 2032])
def test_whole_numbers_are_exact_for_every_last_group_of_scales(K):
    M, N = 260, 516
    xq, xs, w, ws = make_exact(M, K, N, seed=K)
    packed = f8().fp8_repack(w, ws)
    want = product(values(xq, xs, True), values(w, ws, False))[0].half()
    exq, exs, ew, ews = make_exact(M, K, N, E=3, seed=K + 1)
    experts, off = f8().fp8_repack(ew, ews), offsets_of([3, 0, M - 3])
    x = values(exq, exs, True)
    ewant = torch.cat([product(x[:3], values(ew[0], ews[0], False))[0],
                       product(x[3:], values(ew[2], ews[2], False))[0]]).half()
    for plan in PLANS:
        say(f"fp8 last group of scales K={K} plan={plan}")
        Y = f8().fp8_gemm(xq, xs, packed, out="fp16", plan=plan)
        assert torch.equal(Y, want), plan
        Y = f8().fp8_grouped_gemm(exq, exs, experts, off, out="fp16", plan=plan)
        assert torch.equal(Y, ewant), plan


@pytest.mark.parametrize("K", [1024, 4096])
def test_rows_do_not_depend_on_their_neighbours_in_tiles(K):
    """... in whatever place of a tile, where both batches take the same parts of K."""
    N = 256
    xq, xs, w, ws = make(64, K, N, seed=18)
    packed = f8().fp8_repack(w, ws)
    for plan in PLANS[3:]:
        flags = f8().plan_flags_fp8(plan)
        if len({f8().fp8_workspace_bytes(M, N, K, flags) for M in (1, 64)}) > 1:
            continue
        say(f"neighbours K={K} plan={plan}")
        whole = f8().fp8_gemm(xq, xs, packed, plan=plan)
        for row in (0, 37, 63):
            one = f8().fp8_gemm(xq[row:row + 1], xs[row:row + 1], packed, plan=plan)
            assert torch.equal(one[0], whole[row]), (plan, row)
