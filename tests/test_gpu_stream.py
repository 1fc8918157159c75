"""GPU tests of calls with `stream=`: a call on another stream than torch's current one owes
nothing to what the current stream still has to do."""
import pytest

from gpu_helpers import lib, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    lib()


def f8():
    from w4a16_dequant_gemm_amd import fp8
    return fp8


def whole_numbers(M, K, N, seed):
    """An fp8 product whose result is exact: (xq, xs, packed, Y in bf16)."""
    g = torch.Generator().manual_seed(seed)
    xq, w = (torch.randint(-2, 3, (n, K), generator=g).float() for n in (M, N))
    kb, nb = -(-K // 128), -(-N // 128)
    xs, ws = torch.full((M, kb), 0.5), torch.full((nb, kb), 0.25)
    want = (xq.double() @ w.double().t() * 0.125).to(torch.bfloat16).cuda()
    packed = f8().fp8_repack(w.to(E4M3).cuda(), ws.cuda())
    return xq.to(E4M3).cuda(), xs.cuda(), packed, want


def keep_busy(x):
    """Some tens of milliseconds of work for the current stream."""
    for _ in range(30):
        x = x @ x * 1e-3
    return x


def test_first_use_of_a_stream_whose_plan_needs_a_workspace():
    xq, xs, packed, want = whole_numbers(100, 4096, 512, 1)
    assert f8().fp8_workspace_bytes(100, 512, 4096) > 0      # K in parts
    big = torch.rand(4096, 4096, device="cuda")
    keep_busy(big)
    for rep in range(3):
        say(f"stream= with the current stream at work, {rep}")
        side = torch.cuda.Stream()
        Y = torch.full_like(want, float("nan"))
        torch.cuda.synchronize()
        keep_busy(big)
        f8().fp8_gemm(xq, xs, packed, Y=Y, stream=side)
        side.synchronize()
        with torch.cuda.stream(side):
            got = Y.clone()
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_rows_dropped_in_a_chain_on_another_stream():
    """The chain's rows are dropped while the other stream still reads them; the current
    stream then makes and fills memory of the same sizes."""
    from w4a16_dequant_gemm_amd import rowquant
    T, K, N = 512, 4096, 1024
    g = torch.Generator().manual_seed(2)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).cuda()
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    _, _, packed, _ = whole_numbers(1, K, N, 3)
    q, s, _ = rowquant.rmsnorm_quantize_rows(x, w)
    want = f8().fp8_gemm(q, s, packed)
    del q, s
    big = torch.rand(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    for rep in range(5):
        say(f"chain on another stream, {rep}")
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            keep_busy(big)
        q, s, _ = rowquant.rmsnorm_quantize_rows(x, w, stream=side)
        Y = f8().fp8_gemm(q, s, packed, stream=side)
        shape = q.shape
        del q, s
        junk = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda") for _ in range(4)]
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)
        del junk


def test_graphs_that_make_their_own_workspaces():
    """Two graphs captured on one stream with no workspace given, replayed in the other
    order first, with calls outside between the replays."""
    cases = [whole_numbers(100, 4096, 512, 5), whole_numbers(90, 8192, 512, 6)]
    for M, (xq, _, _, want) in zip((100, 90), cases):
        assert f8().fp8_workspace_bytes(M, 512, xq.shape[1]) > 0
    side = torch.cuda.Stream()
    graphs = []
    for xq, xs, packed, want in cases:
        Y = torch.empty_like(want)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            f8().fp8_gemm(xq, xs, packed, Y=Y)
            f8().fp8_gemm(xq, xs, packed, Y=Y)     # the same workspace again
        graphs.append((graph, Y, want))
    for rep in range(3):
        for graph, Y, want in reversed(graphs):
            say(f"replay {rep}")
            Y.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(Y, want), rep
        for xq, xs, packed, want in cases:
            got = f8().fp8_gemm(xq, xs, packed, stream=side)
            torch.cuda.synchronize()
            assert torch.equal(got, want)


def test_inputs_dropped_while_another_stream_still_reads_them():
    from w4a16_dequant_gemm_amd import rowquant
    T, W = 512, 4096
    kept = torch.randn(T, W, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    w = torch.ones(W, dtype=torch.bfloat16, device="cuda")
    want = rowquant.rmsnorm_quantize_rows(kept, w)[:2]
    big = torch.rand(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    for rep in range(5):
        say(f"inputs dropped, {rep}")
        x = kept.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            keep_busy(big)
        q, s, _ = rowquant.rmsnorm_quantize_rows(x, w, stream=side)
        del x
        junk = [torch.full_like(kept, float("nan")) for _ in range(4)]
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(q.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s, want[1])
        del junk
