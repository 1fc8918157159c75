"""Scratch memory of the calls that are several launches (the router, the adapters), without a
GPU: what one call's kernels hand on must be out of reach of any other call's that another
host thread launches between them on the same stream."""
import threading
import weakref

import pytest
import torch

import w4a16_dequant_gemm_amd as w4

from host_fakes import FakeLibrary, fake

DEVICE = torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def on_the_host(monkeypatch):
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *shape, dtype=None, device=None:
                        zeros(*shape, dtype=dtype))
    monkeypatch.setattr(w4, "_on_stream", lambda index, handle: threading.Lock())
    monkeypatch.setattr(w4, "_workspaces", {})
    monkeypatch.setattr(w4, "_retired_workspaces", [])
    monkeypatch.setattr(w4, "_capture_number", lambda handle: None)
    monkeypatch.setattr(torch._C, "_cuda_isCurrentStreamCapturing", lambda: False)


def in_threads(n, f):
    """f() in n threads, one after the other, all alive until the last one is done."""
    got, failed, over = [None] * n, [], threading.Event()

    def work(i, done):
        try:
            got[i] = f()
        except Exception as e:   # shown below: a thread's own would only be printed
            failed.append(e)
        done.set()
        over.wait(60)
    threads = []
    for i in range(n):
        done = threading.Event()
        threads.append(threading.Thread(target=work, args=(i, done)))
        threads[-1].start()
        done.wait(60)
    over.set()
    for t in threads:
        t.join()
    assert not failed
    return got


@pytest.mark.parametrize("stream,handle", [(None, 0), (None, 0x20), ("s", 0x20)])
def test_threads_on_one_stream_share_no_scratch(stream, handle):
    def twice():
        first = w4._scratch(100, DEVICE, stream, handle)
        return first, w4._scratch(1000, DEVICE, stream, handle)
    pairs = in_threads(3, twice) + [twice()]
    for first, again in pairs:
        assert first is again                     # a thread's calls follow one another
    assert len({first.data_ptr() for first, _ in pairs}) == 4


def test_scratch_is_not_the_products_workspace():
    """A product in another thread leaves its parts of sums there, between a call's launches."""
    shared = w4._workspace_at(100, 0, 0x20)
    assert w4._scratch(100, DEVICE, None, 0x20) is not shared
    assert w4._workspace_at(100, 0, 0x20) is shared


def test_scratch_grows_and_goes_with_its_thread():
    kept = []

    def grow():
        first = w4._scratch(1 << 20, DEVICE, None, 0x20)
        larger = w4._scratch((1 << 20) + 1, DEVICE, None, 0x20)
        assert larger is not first and larger.numel() > 1 << 20
        assert w4._scratch(1 << 20, DEVICE, None, 0x20) is larger
        assert w4._scratch(100, DEVICE, None, 0x30) is not larger      # another stream
        kept.append(weakref.ref(larger))
    in_threads(1, grow)
    assert kept[0]() is None                      # nothing keeps what no launch will name again


class Noting(FakeLibrary):
    """Notes the workspace of every call that gets one."""

    def __init__(self, seen):
        self.seen = seen

    def route_workspace_bytes(self, *args):
        return 1 << 17

    lora_workspace_bytes = route_workspace_bytes

    def route_tokens(self, *args):
        self.seen.append(args[-3])
        return 0

    lora_add = route_tokens


def test_calls_of_two_threads_get_scratch_of_their_own(monkeypatch):
    from w4a16_dequant_gemm_amd import lora, route
    from test_boundary_host_route_lora import Buffer
    seen = []
    for module in (route, lora):
        monkeypatch.setattr(module, "_lib", lambda: Noting(seen))
        monkeypatch.setattr(module, "_ws_bytes", {})
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(w4, "_stream_handle", lambda stream: 0)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None:
                        Buffer(*((shape,) if isinstance(shape, int) else shape), dtype=dtype))
    monkeypatch.setattr(torch, "empty_like", lambda like: fake(*like.shape, dtype=like.dtype))
    bf16 = torch.bfloat16

    def both():
        route.route_tokens(fake(100, 16, dtype=torch.float32), 4)
        lora.lora_add(fake(200, 40, dtype=bf16), fake(200, 64, dtype=bf16),
                      fake(3, 8, 64, dtype=bf16), fake(3, 40, 8, dtype=bf16),
                      fake(200, dtype=torch.int32))
    in_threads(2, both)
    # a thread's two calls share, the threads do not
    assert len(seen) == 4 and None not in seen and len(set(seen)) == 2
