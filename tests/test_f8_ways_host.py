"""Every way of the 8-bit float products that the rule takes is one that the GPU tests run (tests/f8ways.py)."""
import math
import random

import pytest

pytest.importorskip("torch")

import f8ways  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    import os

    import gemv_bit_unpack_amd as g

    if not os.path.exists(g.LIB_PATH):
        from gemv_bit_unpack_amd import build

        build.build()
    return g.lib()


def test_every_way_is_tested(lib):
    """Ways that 40000 shapes take, spread over the sizes' logarithms, few rows often; none of them untested."""
    tested = set().union(*(f8ways.ways(lib, *s) for s in f8ways.SHAPES))
    rng, found = random.Random(5), {}
    size = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    for _ in range(40000):
        m = rng.randint(1, 16) if rng.random() < 0.3 else size(1, 8192)
        n, k = size(1, 65536), size(1, 65536)
        for gated in (False, True):
            for way in f8ways.ways(lib, m, n, k, gated):
                found.setdefault(way, (m, n, k, gated))
    assert len(found) >= 50
    missing = {way: shape for way, shape in found.items() if way not in tested}
    assert not missing, missing


@pytest.mark.parametrize("m,d,i,hidden", f8ways.LAYERS)
def test_layers(lib, m, d, i, hidden):
    assert f8ways.writes_hidden(lib, m, d, i) == hidden
