"""GPU: the product of bf16 rows with an MXFP4 matrix: its fp32 sums by norm, and both ends of the scale range.

Tolerances.  A product's sums are K / 32 results of the matrix instruction, added up, and at most 40 more where wavefronts and splits join;
each addition, and the instruction's own of 32 products, counted with a whole step, 2^-23, of a partial sum.  Over a matrix of
independent terms the partial sums' norm is at most the result's, so the error's norm is at most NORM(K) = 2 (K / 32 + 40) 2^-23
of it (2^-14 at K = 7168, where a sum held in bf16 anywhere would be off by 2^-9).  A product of one value, one weight: exact."""
import numpy as np
import pytest
import torch

from oracle import mx4
from ops_util import DEV, gen, host, randn
from test_gpu_mxfp4 import BF, F32, SIZES, matmul, weights

pytestmark = pytest.mark.gpu


def NORM(K):
    return 2 * (K / 32 + 40) * 2.0 ** -23


LONG = [(8, 200, 12288), (9, 200, 8192), (9, 200, 8320), (12, 1000, 9216), (16, 4096, 12288), (16, 40, 28672), (5, 40, 28672)]


@pytest.mark.parametrize("M,N,K", [m for m in SIZES + LONG if m[0] * m[1] >= 64])
def test_fp32_sums(M, N, K):
    print(f"\n[case] matmul_mxfp4 fp32 sums {M}x{N}x{K}", flush=True)
    g = gen(M + N + K)
    x = randn(g, M, K, dtype=BF)
    w, s, W = weights(g, N, K)
    ref = host(x) @ W.T
    err = np.linalg.norm(host(matmul(x, w, s, F32)) - ref) / np.linalg.norm(ref)
    print(f"  error {err:.2e} of {NORM(K):.2e}", flush=True)
    assert err <= NORM(K)


@pytest.mark.parametrize("M", [1, 3, 12, 40, 300])
@pytest.mark.parametrize("ty", [BF, F32])
def test_scales_at_both_ends(M, ty):
    """Every code under the scale bytes 0, 1, 2 (weights below bf16's normal numbers) and 252, 253, 254: a weight past bf16's
    range, 2^128 and above, counts as infinite, which under 253 and 254 only the larger codes are."""
    print(f"\n[case] matmul_mxfp4 scale ends {M} {ty}", flush=True)
    K = 256
    byte = np.repeat([0, 1, 2, 252, 253, 254], 16)
    code = np.tile(np.arange(16), 6)
    N = len(byte)
    at = np.arange(N) * 37 % K
    w = np.zeros((N, K // 2), dtype=np.uint8)
    w[np.arange(N), at // 2] = code << (4 * (at % 2))
    s = np.broadcast_to(byte[None, :, None], (K // 128, N, 4)).astype(np.uint8).copy()
    value = mx4.TABLE[code] * 2.0 ** (byte - 127.0)
    assert np.array_equal(mx4.values(w, s)[np.arange(N), at], value)
    value = np.where(abs(value) >= 2.0 ** 128, np.copysign(np.inf, value), value)
    assert np.isfinite(value[byte <= 252]).all()
    for rows, up in ((byte <= 2, 100), (byte >= 252, -100)):
        x = torch.exp2(torch.full((M, K), float(up), device=DEV)) * (1 + 0.5 * (torch.arange(M, device=DEV)[:, None] % 2))
        x[::3] *= -1
        out = host(matmul(x.to(BF), torch.tensor(w[rows], device=DEV), torch.tensor(s[:, rows], device=DEV).contiguous(), ty))
        want = host(x)[:, at[rows]] * value[rows]
        assert np.isfinite(want).any() and np.array_equal(out, want), np.argwhere(out != want)[:5].tolist()
