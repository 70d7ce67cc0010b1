"""Which form of the MXFP4 product runs, seen from its workspace (no GPU): a stream of W needs none, tiles of few rows split K."""
import pytest

from mixture_experts_layer_33_amd import _lib


def workspace(M, N, K):
    return _lib.lib().moe_matmul_mxfp4_workspace_bytes(M, N, K)


@pytest.mark.parametrize("M,K", [(1, 128), (8, 8192), (8, 28672), (9, 8192), (16, 2048), (16, 8192)])
def test_streams(M, K):
    assert workspace(M, 512, K) == 0


@pytest.mark.parametrize("M,K", [(9, 8320), (12, 9216), (16, 28672), (17, 8192)])
def test_rows_that_do_not_stay_in_registers_go_in_tiles(M, K):
    """16 x 512 x 9216: 14.5 us as a stream that reads x again for every unit, 9.7 in tiles."""
    assert workspace(M, 512, K) >= 2 * M * 512 * 4
