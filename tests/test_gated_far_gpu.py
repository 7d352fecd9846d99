"""The gated block's values far from zero on the GPU, against the formulas in
64 bits (oracle/gated.py): gates whose sigmoid is below the smallest normal
FP32 number, with factors that bring the result back into range."""
import numpy as np
import pytest

import dense_gemm_mgemm_amd as mg  # noqa: F401
from oracle import gated
from test_gated_gpu import EPS, TINY, Block, h, rounded, say, wide  # noqa: F401

pytestmark = pytest.mark.gpu

# e^g is a normal FP32 number down to g = -87.3 and a subnormal one down to -103.
FAR = [-19.5, -20.5, -60.0, -86.0, -87.5, -88.0, -90.0, -99.5, -103.5, -110.0, -130.0, -150.0]


@pytest.mark.parametrize("again", [False, True])
def test_gradients_of_closed_gates(h, again):  # noqa: F811
    """dG and dU of a gate that is shut, under gradients and values as large as BF16 holds them: off by the rounding to
    BF16 and 1e-5 of FP32 arithmetic (the products with an identity add nothing), with no absolute slack."""
    say("gated_backward far gates", again)
    n = len(FAR)
    g = np.repeat(rounded(np.array(FAR), "bf16")[:, None], n, 1)
    u, dz = np.full((n, n), 2.0 ** 30), np.zeros((n, n))
    big = 2.0 ** np.array([0.0, 20.0, 60.0, 90.0, 95.0, 40.0, 80.0, 95.0, 93.0, 95.0, 95.0, 95.0])
    dz[np.arange(n), np.arange(n)] = rounded(big * np.linspace(1.0, 1.9, n), "bf16")
    if again:
        # X is the identity, so G and U are the weights' rows.
        b = Block(h, "row", n, n, n, "bf16", np.eye(n), g, u)
        outs = b.backward(wide(dz, n, "bf16"), dx=False)
        _, dwg, dwu = b.grads(outs)
    else:
        b = Block(h, "row", n, n, n, "bf16", np.eye(n), np.zeros((n, n)), np.zeros((n, n)))
        _, dwg, dwu = b.grads(b.backward(*(wide(v, n, "bf16") for v in (dz, g, u))))
    dg, du = gated.pointwise(g, u, dz)
    assert np.abs(dg).max() < 2.0 ** 127              # representable, all of them
    for got, ref in ((dwg, dg), (dwu, du)):
        assert np.isfinite(got).all()
        off = np.abs(got - ref) > (EPS["bf16"] + 1e-5) * np.abs(ref) + TINY["bf16"]
        assert not off.any(), [(FAR[i], got[i, j], ref[i, j]) for i, j in np.argwhere(off)[:4]]


def test_one_closed_gate_leaves_the_others_bits(h):  # noqa: F811
    """A wave that holds a closed gate takes another form of the sigmoid: its other outputs keep their bits."""
    n = 64
    rng = np.random.default_rng(6)
    g, u, dz = (rounded(v, "bf16") for v in (rng.uniform(-19.9, 19.9, (n, n)), rng.standard_normal((n, n)),
                                             rng.standard_normal((n, n))))
    b = Block(h, "row", n, n, n, "bf16", np.eye(n), np.zeros((n, n)), np.zeros((n, n)))
    _, dwg, dwu = b.grads(b.backward(*(wide(v, n, "bf16") for v in (dz, g, u))))
    g[::7, 5] = -95.0
    _, awg, awu = b.grads(b.backward(*(wide(v, n, "bf16") for v in (dz, g, u))))
    keep = np.ones((n, n), bool)
    keep[::7, 5] = False
    assert np.array_equal(dwg[keep], awg[keep]) and np.array_equal(dwu[keep], awu[keep])
