"""VQLinear's workspaces: each call has one of its own (no sharing between threads or captured graphs, none of it kept),
and their contents need no initialisation.

On the host the library's launches are replaced by ones that note the workspace they are given; on the GPU a captured
call is replayed after a larger one on its stream.
"""
import threading

import pytest

torch = pytest.importorskip("torch")

N, K = 2048, 2048   # 2^19 weight vectors: both paths take a workspace from 8 rows on


@pytest.fixture(scope="module")
def vq():
    import os

    import gemv_bit_unpack_amd as g

    if not os.path.exists(g.LIB_PATH):
        from gemv_bit_unpack_amd import build

        build.build()
    g.lib()
    return g


def _layer(vq, device):
    desc = vq.make_desc(N, K, 8, 16, 8)
    g = torch.Generator().manual_seed(1)
    packed = torch.randint(0, 256, (vq.packed_bytes(desc),), generator=g, dtype=torch.uint8)
    book = lambda n: (torch.randn((n, 8), generator=g) * 0.02).half()
    return vq.VQLinear(desc, *(t.to(device) for t in (packed, book(1 << 16), book(256), torch.ones(N).half())))


class _Noted:
    def __init__(self, real):
        self.real, self.seen, self.barrier = real, [], None

    def __getattr__(self, name):
        if name not in ("vq_gemv_ws", "vq_gemm_ws"):
            return getattr(self.real, name)

        def launch(*args):
            self.seen.append((args[11].value, args[12]))
            if self.barrier is not None:
                self.barrier.wait(60)
            return 0

        return launch


@pytest.fixture
def noted(vq, monkeypatch):
    import ctypes

    lib = _Noted(vq.lib())
    monkeypatch.setattr(vq, "lib", lambda: lib)
    monkeypatch.setattr(vq, "_dev_ptr", lambda t, what, dtypes=None: None if t is None else ctypes.c_void_p(t.data_ptr()))
    monkeypatch.setattr(vq, "_stream_ptr", lambda device: None)
    return lib


@pytest.mark.parametrize("m", [8, 40])
def test_calls_of_two_threads_share_nothing(vq, noted, m):
    layer = _layer(vq, "cpu")
    layer(torch.zeros((m, K), dtype=torch.bfloat16))
    noted.seen.clear()
    noted.barrier = threading.Barrier(2)
    failed = []

    def work():
        try:
            layer(torch.zeros((m, K), dtype=torch.bfloat16))
        except Exception as e:  # noqa: BLE001 - told by the assertion below
            failed.append(e)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and len(noted.seen) == 2, failed
    (a, na), (b, nb) = noted.seen
    assert na > 0 and (a + na <= b or b + nb <= a)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [8, 40])
def test_larger_call_after_a_capture(vq, m):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    layer = _layer(vq, "cuda")
    make = lambda rows, seed: torch.randn((rows, K), generator=torch.Generator(device="cuda").manual_seed(seed),
                                          device="cuda").bfloat16()
    st = torch.cuda.Stream()
    x = make(m, 1)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        layer(x)  # as a warm-up before a capture does
    st.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=st):
        y = layer(x)
    with torch.cuda.stream(st):
        layer(make(3000, 2))
        fill = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                for n in (1 << 12, 1 << 15, m * K * 2, 1 << 18, 1 << 20, 1 << 22, 1 << 24) for _ in range(4)]
    st.synchronize()
    for k in range(3):
        x.copy_(make(m, 10 + k))
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, layer(x)), k
        assert all(bool((f == 255).all()) for f in fill), k
    del fill  # the next calls' workspaces hold 255 in every byte
    with torch.cuda.stream(st):
        again = layer(x)
    st.synchronize()
    assert torch.equal(again, y)
