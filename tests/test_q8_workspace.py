"""The layers' workspaces: each call has one of its own, so that calls of other threads, captured calls that are replayed
later and larger calls after them never share scratch memory.

On the host the library's launches are replaced by ones that note the workspace they are given; on the GPU the sharing
that would show is set up in earnest.
"""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def vq():
    import os

    import gemv_bit_unpack_amd as g

    if not os.path.exists(g.LIB_PATH):
        from gemv_bit_unpack_amd import build

        build.build()
    g.lib()
    return g


# ---------------------------------------------------------------- on the host


class _Noted:
    """The library with its launches replaced: they note (workspace, bytes) and meet at a barrier if there is one."""

    LAUNCHES = {"vq_q8_linear": (11, 12), "vq_q8_gemm": (10, 11), "vq_q8_experts": (16, 17)}

    def __init__(self, real):
        self.real, self.seen, self.barrier = real, [], None

    def __getattr__(self, name):
        if name not in self.LAUNCHES:
            return getattr(self.real, name)
        at, size = self.LAUNCHES[name]

        def launch(*args):
            self.seen.append((args[at], args[size]))
            if self.barrier is not None:
                self.barrier.wait(60)
            return 0

        return launch


@pytest.fixture
def noted(vq, monkeypatch):
    lib = _Noted(vq.lib())
    monkeypatch.setattr(vq.q8, "lib", lambda: lib)
    monkeypatch.setattr(vq.q8, "_device", lambda t, what: -1)
    monkeypatch.setattr(vq.q8, "_stream", lambda dev: 0)
    return lib


def _calls(vq):
    """(name, a call with `m` rows that needs a workspace) of each layer call."""
    lin = vq.Q8Linear(torch.zeros((64, 200), dtype=torch.int8), torch.ones(64))
    cut = vq.Q8Linear(torch.zeros((64, 65536), dtype=torch.int8), torch.ones(64))
    exp = vq.Q8Experts(torch.zeros((2, 64, 128), dtype=torch.int8), torch.ones((2, 64)),
                       torch.zeros((2, 128, 32), dtype=torch.int8), torch.ones((2, 128)))
    zeros = lambda m, k, dt=torch.float16: torch.zeros((m, k), dtype=dt)
    return [("linear", lambda m: lin(zeros(m, 200))),
            ("products of 8-bit tokens", lambda m: cut.forward_q8(zeros(m, 65536, torch.int8), torch.ones(m))),
            ("experts", lambda m: exp(zeros(m, 128), zeros(m, 2, torch.int32), torch.ones((m, 2))))]


class _Made(torch.utils._python_dispatch.TorchDispatchMode):
    """Keeps every tensor that an operator makes."""

    def __init__(self):
        super().__init__()
        self.tensors = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if isinstance(out, torch.Tensor):
            self.tensors.append(out)
        return out


def test_each_call_makes_its_own(vq, noted):
    kept = []
    for name, call in _calls(vq):
        for m in (70, 90, 70):  # grown and shrunk again
            with _Made() as made:
                call(m)
            kept.append(made.tensors)
            at, nbytes = noted.seen[-1]
            assert nbytes > 0, name
            assert any(t.data_ptr() == at and t.numel() * t.element_size() >= nbytes for t in made.tensors), (name, m)


def test_calls_of_two_threads_share_nothing(vq, noted):
    for name, call in _calls(vq):
        noted.seen.clear()
        noted.barrier = threading.Barrier(2)
        failed = []

        def work():
            try:
                call(70)
            except Exception as e:  # noqa: BLE001 - told by the assertion below
                failed.append(e)

        threads = [threading.Thread(target=work) for _ in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        noted.barrier = None
        assert not failed and len(noted.seen) == 2, (name, failed)
        (a, na), (b, nb) = noted.seen
        assert a + na <= b or b + nb <= a, name


# ---------------------------------------------------------------- on the GPU


@pytest.fixture
def gpu(vq):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return vq


def _layers(vq):
    """(name, layer call, x of m rows) of a linear layer and an expert layer."""
    g = np.random.default_rng(17)
    w = lambda *s: torch.from_numpy(np.clip(np.rint(g.standard_normal(s) * 40), -127, 127).astype(np.int8)).cuda()
    sc = lambda *s: torch.from_numpy(g.uniform(0.5, 1.5, s).astype(np.float32) * np.float32(6e-4)).cuda()
    lin = vq.Q8Linear(w(300, 7000), sc(300))
    exp = vq.Q8Experts(w(4, 256, 700), sc(4, 256), w(4, 700, 128), sc(4, 700))

    def x(m, k, seed):
        return torch.randn((m, k), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").half()

    def experts(v):
        m = v.shape[0]
        r = torch.arange(m, device="cuda", dtype=torch.int32)
        return exp(v, torch.stack([r % 4, (r + 1) % 4], dim=1).contiguous(), torch.full((m, 2), 0.5, device="cuda"))

    return [("linear", lin, lambda m, seed: x(m, 7000, seed)), ("experts", experts, lambda m, seed: x(m, 700, seed))]


@pytest.mark.gpu
def test_larger_call_after_a_capture(gpu):
    """A captured call, then a larger one on its stream, then tensors of every size its scratch memory could go to: replays
    give the captured call's results and leave the tensors alone."""
    for name, call, make in _layers(gpu):
        st = torch.cuda.Stream()
        x = make(40, 1)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            call(x)  # as a warm-up before a capture does
        st.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            y = call(x)
        with torch.cuda.stream(st):
            call(make(3000, 2))
            fill = [torch.full((n,), 7, dtype=torch.uint8, device="cuda")
                    for n in (1 << 10, 40 * 128, 40 * 768, 1 << 16, 40 * 7040, 1 << 19, 1 << 20, 1 << 21, 1 << 23) for _ in range(4)]
        st.synchronize()
        for k in range(3):
            x.copy_(make(40, 10 + k))
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, call(x)), (name, k)
            assert all(bool((f == 7).all()) for f in fill), (name, k)


@pytest.mark.gpu
def test_two_graphs_at_once(gpu):
    """Two graphs captured on the same stream and replayed on two: each gives its own results."""
    for name, call, make in _layers(gpu):
        xs = [make(500, 3), make(500, 4)]
        want = [call(x) for x in xs]
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        graphs, out = [], []
        for x in xs:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=st):
                out.append(call(x))
            graphs.append(gr)
        streams = [torch.cuda.Stream() for _ in graphs]
        for _ in range(3):
            for o in out:
                o.zero_()
            torch.cuda.synchronize()
            for _ in range(8):
                for s, gr in zip(streams, graphs):
                    with torch.cuda.stream(s):
                        gr.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), name


@pytest.mark.gpu
def test_two_threads_on_one_stream(gpu):
    for name, call, make in _layers(gpu):
        xs = [make(33, 5), make(47, 6)]
        want = [call(x) for x in xs]
        torch.cuda.synchronize()
        wrong = []

        def work(x, y):
            wrong.extend(k for k in range(200) if not torch.equal(call(x), y))

        threads = [threading.Thread(target=work, args=a) for a in zip(xs, want)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not wrong, (name, len(wrong))


def test_one_token_without_a_workspace(vq, noted):
    """One token up to ONE_MAX_K columns takes none, a longer row or a second token does; the library refuses its absence."""
    for k, m in ((200, 1), (vq.q8.ONE_MAX_K, 1), (vq.q8.ONE_MAX_K + 1, 1), (200, 2)):
        lay = vq.Q8Linear(torch.zeros((3, k), dtype=torch.int8), torch.ones(3))
        lay(torch.zeros((m, k)))
        assert (noted.seen[-1] == (None, 0)) == (m == 1 and k <= vq.q8.ONE_MAX_K), (k, m)
    p = 1 << 20
    linear = lambda m, k, ws, nbytes: vq.lib().vq_q8_linear(m, 3, k, p, 0, k, p, p, None, p, 0, ws, nbytes, None)
    assert linear(1, vq.q8.ONE_MAX_K + 1, None, 0) == vq.VQ_ERR_NULL
    assert linear(2, 200, None, 0) == vq.VQ_ERR_NULL
    assert linear(1, 200, p, 16) == vq.VQ_ERR_BUFFER_SIZE     # one that is given is checked
    assert linear(1, 200, p + 16, 1 << 20) == vq.VQ_ERR_ALIGN


@pytest.mark.gpu
@pytest.mark.parametrize("k", [1, 200, 48128])
def test_one_token_without_a_workspace_same_bits(gpu, k):
    g = torch.Generator(device="cuda").manual_seed(k)
    w = gpu.q8_pad(torch.randint(-127, 128, (50, k), generator=g, device="cuda", dtype=torch.int8))
    sw = torch.rand((50,), generator=g, device="cuda")
    x = torch.randn((1, k), generator=g, device="cuda")
    y = gpu.q8_linear(x, w, sw, None, None)
    q, s = gpu.q8_quantize(x)
    assert torch.equal(y, gpu.q8_gemm(q, s, w, sw, None, k, y_dtype=torch.float32))
