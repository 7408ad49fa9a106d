"""Host-only checks of the norms' size queries at the ends of their ranges."""

import pytest

from tests.test_abi_host import _lib

MOST = (1 << 31) - 1


@pytest.mark.parametrize("D", [1, 2, 37, 96, 256, 257, 1001, 1024, 4096, 8192, 16384])
def test_layer_norm_gradients_of_the_most_tokens(D):
    """A partial row per block and weight: as many at any number of tokens that fills the GPU."""
    ops, _ = _lib()
    want = ops.layer_norm_bwd_workspace_size(1 << 24, D)
    assert 0 < want <= 2 * 148 * 4 * D * 4 + 256
    for n in (MOST, MOST - 1, MOST - 6, MOST - 7, MOST - 8, 1 << 30):
        assert ops.layer_norm_bwd_workspace_size(n, D) == want, n
