"""The page pool with the most sequences that it takes, each named once or more in the lists, against the plain reference."""
import numpy as np
import pytest

from test_gpu_kv_pool import make, setup  # noqa: F401

pytestmark = pytest.mark.gpu
N = 65536


def test_the_most_sequences():
    rng = np.random.default_rng(1)
    g = make(N, 3, 180000, 16, lens=rng.integers(0, 40, N), layers=((1, 16),))
    g.free(list(rng.integers(-3, N + 3, N)), list(rng.integers(0, 30, N)), list(rng.integers(0, 50, N)))
    g.reserve(list(rng.integers(-1, 6, N)))
    g.compact()
    g.free(list(range(0, N, 3)))
    g.fork(list(rng.integers(0, N, N)), list(rng.permutation(N)))
    g.reserve([1] * N)
    g.ref.check()
    g.compact()
