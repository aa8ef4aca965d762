"""CPU checks of the dense products' documented limits, to the last size inside them.  No call here reaches a kernel
launch: where a size is inside, a misaligned result is refused next."""
import pytest

from combine_get_dispatch_histogram_amd import _lib

EUNSUPPORTED = _lib.MIEP_EUNSUPPORTED
MOST = 2 ** 31 - 2 ** 16


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from combine_get_dispatch_histogram_amd import build
        build.build()
    return _lib.load()


@pytest.mark.parametrize("n,k", [(1 << 20, 64), (64, 1 << 20), (1 << 21, 1 << 21), (136, 8)])
def test_tiles_of_a_dense_product(lib, n, k):
    rows = min(32 * (MOST // (max(n, k) // 128 + 1) - 2) + 31, MOST)
    assert (rows // 32 + 2) * (max(n, k) // 128 + 1) <= MOST
    for at, word in ((rows, b"16"), (rows + 1, b"tiles" if rows < MOST else b"rows")):
        assert lib.miep_linear(16, at, 16, n, k, None, 0, None, None, 8, 0, None) == EUNSUPPORTED and word in lib.miep_last_error()
        assert lib.miep_linear_dgrad(16, at, 16, n, k, 8, None) == EUNSUPPORTED and word in lib.miep_last_error()
        assert lib.miep_linear_wgrad(16, 16, at, n, k, 1, 0, 8, None) == EUNSUPPORTED and word in lib.miep_last_error()


def test_tiles_of_a_weights_gradient(lib):
    for n, k in (((1 << 19) + 8, 1 << 19), (1 << 19, (1 << 19) + 8), (1 << 21, 1 << 18)):
        assert -(-n // 128) * -(-k // 128) > 2 ** 24
        assert lib.miep_linear_wgrad(16, 16, 64, n, k, 1, 0, 16, None) == EUNSUPPORTED and b"2^24" in lib.miep_last_error()
