"""Infinite weights in the gated block's recomputed backward pass on the GPU:
the rows and columns of zeros that copies of operands are padded with stay
zero, so the answer does not depend on whether an operand was copied."""
import numpy as np
import pytest

import dense_gemm_mgemm_amd as mg  # noqa: F401
from test_gated_gpu import Block, h, say, wide  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size,ksplit", [(128, 1), (128, 3), (256, 1), (256, 3)])
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("pad", [0, 3])
def test_infinite_weight(h, layout, pad, size, ksplit):  # noqa: F811
    """One infinite entry of Wu: U and dG are infinite in its column, with the sign of dZ U s (1 + G (1 - s)) > 0, so
    that column of dWg is X^T times infinities of one sign and dX, dWu follow; nothing in it is a NaN but dX where
    infinities meet.  Every other column is what it was."""
    say("gated_backward infinite weight", layout, pad, size, ksplit)
    M, N, K = 70, 72, 200
    n0 = 17
    rng = np.random.default_rng(8)
    # Positive X, weights and dZ: G > 0, so the derivative is positive.
    x, wg, wu, dz = (rng.integers(1, 3, s) / 8 for s in ((M, K), (K, N), (K, N), (M, N)))

    def grads():
        b = Block(h, layout, M, N, K, "bf16", x, wg, wu, pad)
        try:
            mg.mgemm_set_gated_tile(h, 0, size, ksplit)
            return b.grads(b.backward(wide(dz, N + pad, "bf16")))
        finally:
            mg.mgemm_set_gated_tile(h, 0)
    before = grads()
    wu[30, n0] = np.inf
    dx, dwg, dwu = grads()
    assert np.array_equal(np.delete(dwg, n0, 1), np.delete(before[1], n0, 1))
    assert np.array_equal(dwu, before[2])             # dU does not depend on U
    assert (dwg[:, n0] == np.inf).all()
    assert (dx == np.inf).all()
