"""The recomputed backward pass in each tile and split on the GPU: against the
oracle's gradients, and bit for bit against the pass that is given the same G and
U; and the range of FP16's dG and dU."""
import numpy as np
import pytest
import torch

import dense_gemm_mgemm_amd as mg
from oracle import gated
from test_gated_gpu import Block, backward_bounds, h, ints, rounded, say, wide  # noqa: F401

pytestmark = pytest.mark.gpu


def force(h, size, ksplit):  # noqa: F811
    mg.mgemm_set_gated_tile(h, 0, size, ksplit)


# Tails of the contraction, edges in both directions, several tiles each way; odd strides copy and pad the operands.
@pytest.mark.parametrize("size", [128, 256])
@pytest.mark.parametrize("ksplit", [1, 2, 5, 32])
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("M,N,K,pad", [(300, 424, 616, 0), (130, 520, 1096, 0), (65, 193, 515, 3)])
def test_every_tile(h, size, ksplit, layout, M, N, K, pad):  # noqa: F811
    say("gated again tile", size, ksplit, layout, M, N, K, pad)
    rng = np.random.default_rng(size + ksplit + M)
    # Quarters of integers: the sums are exact in any order, so G and U are rounded as if stored.
    x, wg, wu = ints(rng, (M, K), 2) / 4, ints(rng, (K, N), 3) / 4, ints(rng, (K, N), 3) / 4
    for dtype in ("bf16", "f16"):
        dz = rounded(rng.standard_normal((M, N)), dtype)
        g, u = rounded(x @ wg, dtype), rounded(x @ wu, dtype)
        assert (np.abs(x @ wg) < 2.0 ** 20).all()
        b = Block(h, layout, M, N, K, dtype, x, wg, wu, pad)
        zd, gd, ud = (wide(v, N + pad, dtype) for v in (dz, g, u))
        stored = b.backward(zd, gd, ud)
        try:
            force(h, size, ksplit)
            again = b.backward(zd)
        finally:
            force(h, 0, 0)
        torch.cuda.synchronize()
        for a, c in zip(again, stored):
            assert torch.equal(a, c)
        for a, (y, lim) in zip(b.grads(again), backward_bounds(x, wg, wu, g, u, dz, dtype)):
            assert (np.abs(a - y) <= lim).all(), np.abs(a - y).max()


# Sizes whose time model takes the 256 tile, and ranges, for the recomputed pair.
@pytest.mark.parametrize("M,N,K", [(2048, 2304, 1000), (64, 1024, 8192), (100, 250, 4100)])
@pytest.mark.parametrize("layout", ["row", "col"])
def test_larger(h, layout, M, N, K):  # noqa: F811
    say("gated again larger", layout, M, N, K)
    gen = torch.Generator(device="cuda").manual_seed(M)

    def pick(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda").double()
    x, wg, wu, dz = pick(-1, 1, M, K), pick(-1, 1, K, N) / 8, pick(-1, 1, K, N) / 8, pick(-8, 8, M, N) / 8
    b = Block(h, layout, M, N, K, "bf16", x, wg, wu)
    g, u = (x @ wg).bfloat16(), (x @ wu).bfloat16()   # sums of up to 8192 eighths: exact in FP32
    zd = dz.bfloat16()
    again, stored = b.backward(zd), b.backward(zd, g, u)
    torch.cuda.synchronize()
    for a, c in zip(again, stored):
        assert torch.equal(a, c)


def test_range_of_fp16(h):  # noqa: F811
    """dG and dU are FP16 matrices between the two stages: beyond 65504 they are infinite and below 2^-25 zero, also
    where the gradients that they lead to would be representable; BF16 holds both."""
    n = 64
    x, w = np.eye(n), np.eye(n)
    g = np.zeros((n, n))                              # s = 1/2: dG = dZ U / 2, dU = 0
    for dtype in ("f16", "bf16"):
        u, dz = np.full((n, n), 1024.0), np.zeros((n, n))
        dz[0, 0], dz[1, 1], dz[2, 2] = 128.0, 96.0, 2.0 ** -14
        u[2, 2] = 2.0 ** -12
        b = Block(h, "row", n, n, n, dtype, x, w / 64, w / 64)
        dx, dwg, _ = b.grads(b.backward(*(wide(v, n, dtype) for v in (dz, g, u))))
        dg, _ = gated.pointwise(g, u, dz)
        assert dg[0, 0] == 65536.0 and dg[1, 1] == 49152.0 and dg[2, 2] == 2.0 ** -27
        # 65536 / 64 = 1024 would be representable in dX.
        assert dx[0, 0] == (np.inf if dtype == "f16" else 1024.0) and dx[1, 1] == 768.0
        assert dwg[0, 0] == (np.inf if dtype == "f16" else 65536.0)
        assert dwg[2, 2] == (0.0 if dtype == "f16" else 2.0 ** -27)
