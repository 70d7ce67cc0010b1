"""moe_matmul_fp8 takes rows of any length whose operands stay below 2^32 elements: its 32-bit offsets are row x K bytes of one
operand.  Statuses from the host's checks before any launch (no GPU), and results on the GPU."""
import pytest
import torch

import mixture_experts_layer_33_amd as moe
from mixture_experts_layer_33_amd import _lib
from ops_util import DEV, gen

FAKE = 0x1000
L = _lib.lib


def mm(M, N, K, a=FAKE):
    return L().moe_matmul_fp8(a, FAKE, FAKE, FAKE, M, N, K, _lib.MOE_BF16, FAKE, FAKE, 1 << 40, None)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1 << 23), (511, 511, 1 << 23), (3, 5, (1 << 24) + 128), (1, 1, (1 << 31) - 128)])
def test_long_rows_are_taken(M, N, K):
    assert mm(M, N, K, a=None) == _lib.MOE_ERR_NULL                    # the sizes passed: the missing operand is what is wrong
    assert L().moe_matmul_fp8_workspace_bytes(M, N, K) % 256 == 0


@pytest.mark.parametrize("M,N,K", [(512, 1, 1 << 23), (1, 512, 1 << 23), (1, 1, 1 << 31), (1, 1, (1 << 23) + 64)])
def test_too_many_elements_are_refused(M, N, K):
    assert mm(M, N, K) == _lib.MOE_ERR_SHAPE


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(3, 5, 1 << 23), (40, 130, (1 << 23) + 128)])
@pytest.mark.parametrize("ty", [torch.bfloat16, torch.float32])
def test_long_rows(M, N, K, ty):
    """Small integers at a few places of every row, the first and the last among them: the sums are exact in any order."""
    print(f"\n[case] matmul_fp8 long rows {M}x{N}x{K} {ty}", flush=True)
    g = gen(M)
    at = torch.tensor([0, 1, 127, 128, K // 2, K - 129, K - 2, K - 1], device=DEV)
    part = {n: torch.randint(-2, 3, (n, len(at)), generator=g, device=DEV).float() for n in (M, N)}

    def rows(n):
        c = torch.zeros(n, K, dtype=torch.uint8, device=DEV)
        c[:, at] = part[n].to(torch.float8_e4m3fn).view(torch.uint8)
        return c

    out = torch.full((M, N), 99, dtype=ty, device=DEV)
    moe.moe_matmul_fp8(rows(M), torch.ones(K // 128, M, device=DEV), rows(N), torch.ones((N + 127) // 128, K // 128, device=DEV), out,
                       moe.matmul_fp8_workspace(M, N, K, DEV))
    torch.cuda.synchronize()
    assert torch.equal(out.cpu().double(), part[M].cpu().double() @ part[N].cpu().double().T)
