"""The gated block's oracle against differences, and the entry points'
refusals (no GPU: every call is refused before anything is enqueued)."""
import ctypes

import numpy as np
import pytest

import dense_gemm_mgemm_amd as mg
from oracle import gated


def test_gradients_are_differences():
    rng = np.random.default_rng(1)
    M, N, K = 4, 5, 6
    x, wg, wu, dz = (rng.standard_normal(s) for s in ((M, K), (K, N), (K, N), (M, N)))
    _, g, u = gated.forward(x, wg, wu)
    grads = gated.backward(x, wg, wu, g, u, dz)
    step = 1e-6
    for which, (v, d) in enumerate(zip((x, wg, wu), grads)):
        for i in np.ndindex(*v.shape):
            args = [a.copy() for a in (x, wg, wu)]
            args[which][i] += step
            hi = (gated.forward(*args)[0] * dz).sum()
            args[which][i] -= 2 * step
            lo = (gated.forward(*args)[0] * dz).sum()
            # Central differences: step^2 of the third derivative, and 2^-53 of the sum over the step.
            assert abs((hi - lo) / (2 * step) - d[i]) < 1e-7


def test_far_values():
    g = np.array([-800.0, -40.0, 0.0, 40.0, 800.0])
    dg, du = gated.pointwise(g, np.ones(5), np.ones(5))
    assert np.allclose(dg, [0, -39 * np.exp(-40), 0.5, 1, 1], rtol=1e-12)
    assert np.allclose(du, [0, -40 * np.exp(-40), 0, 40, 800], rtol=1e-12)


INVALID, UNSUPPORTED = mg.MGEMM_ERR_INVALID_ARG, mg.MGEMM_ERR_UNSUPPORTED
_fake = ctypes.create_string_buffer(4096)           # stands for a handle and for pointers: never read


def _p(offset=0):
    return ctypes.addressof(_fake) // 16 * 16 + 16 + offset


def workspace(layout=0, M=4, N=8, K=16, x=_p(), ldx=16, wg=_p(), wu=_p(), ldw=8, dtype=2, backward=0, stored=0):
    out = ctypes.c_int64(-1)
    st = mg.load().mgemm_gated_workspace(layout, M, N, K, x, ldx, wg, wu, ldw, dtype, backward, stored,
                                         ctypes.byref(out))
    return st, out.value


def test_workspace_sizes():
    # Aligned operands: nothing forward, dG and dU (4 x 8 each, 256-byte pieces and a start's slack) backward.
    assert workspace() == (0, 0)
    assert workspace(backward=1, stored=1) == (0, 3 * 256)
    assert workspace(backward=1, stored=0) == (0, 3 * 256)
    # A copy is 64 x 64 values.  An odd stride or base: X is copied; odd weights: both weights are.
    copy = 64 * 64 * 2
    assert workspace(ldx=17) == (0, copy + 256)
    assert workspace(x=_p(2)) == (0, copy + 256)
    assert workspace(wu=_p(4)) == (0, 2 * copy + 256)
    # A length that is not a multiple of 8 along an output axis.
    assert workspace(N=7) == (0, 2 * copy + 256)
    assert workspace(layout=1, N=7, ldw=16) == (0, 0)
    assert workspace(K=15)[1] == 0                                    # the contraction's tail: in place
    # dW's rows: X is copied, and dG and dU (64 x 8) are padded as its rows are.
    assert workspace(K=15, backward=1, stored=1) == (0, copy + 2 * 1024 + 256)
    assert workspace(M=0, backward=1) == (0, 0)
    assert mg.load().mgemm_gated_workspace(0, 4, 8, 16, _p(), 16, _p(), _p(), 8, 2, 0, 0, None) == INVALID


@pytest.mark.parametrize("bad,status", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(layout=2), INVALID),
    (dict(dtype=3), INVALID), (dict(dtype=0), UNSUPPORTED), (dict(ldx=15), INVALID), (dict(ldw=7), INVALID),
    (dict(layout=1, ldw=15), INVALID), (dict(M=1 << 59), INVALID), (dict(N=1 << 61, ldw=1 << 61), INVALID)])
def test_common_refusals(bad, status):
    assert workspace(**bad)[0] == status
    a = dict(layout=0, M=4, N=8, K=16, ldx=16, ldw=8, dtype=2)
    a.update(bad)
    assert forward(**a) == status
    assert backward(**a) == status


def forward(layout=0, M=4, N=8, K=16, x=_p(), ldx=16, wg=_p(), wu=_p(), ldw=8, z=_p(), ldz=8, g=_p(), u=_p(), ldg=8,
            dtype=2, work=None, size=0, h=_p()):
    return mg.load().mgemm_gated_forward(h, layout, M, N, K, x, ldx, wg, wu, ldw, z, ldz, g, u, ldg, dtype, work, size,
                                         None)


def backward(layout=0, M=4, N=8, K=16, x=_p(), ldx=16, wg=_p(), wu=_p(), ldw=8, g=_p(), u=_p(), ldg=8, dz=_p(), lddz=8,
             dx=_p(), lddx=16, dwg=_p(), dwu=_p(), lddw=None, beta=0.0, dtype=2, work=None, size=0, h=_p()):
    lddw = (8 if layout == 0 else 16) if lddw is None else lddw
    return mg.load().mgemm_gated_backward(h, layout, M, N, K, x, ldx, wg, wu, ldw, g, u, ldg, dz, lddz, dx, lddx, dwg,
                                          dwu, lddw, beta, dtype, work, size, None)


@pytest.mark.parametrize("bad", [dict(h=None), dict(z=None), dict(x=None), dict(wg=None), dict(wu=None), dict(g=None),
                                 dict(u=None), dict(ldz=7), dict(ldg=7), dict(ldx=17),
                                 dict(ldx=17, work=_p(), size=511)])
def test_forward_refusals(bad):
    assert forward(**bad) == INVALID


@pytest.mark.parametrize("bad", [dict(h=None), dict(dz=None), dict(x=None), dict(wg=None), dict(wu=None), dict(g=None),
                                 dict(u=None), dict(dwg=None), dict(dwu=None), dict(lddz=7), dict(ldg=7),
                                 dict(lddx=15), dict(lddw=7), dict(layout=1, ldw=16, lddw=15),
                                 dict(), dict(work=_p(), size=767), dict(g=None, u=None, x=None, work=_p(), size=4096)])
def test_backward_refusals(bad):
    # (An empty dict: no workspace where dG and dU need one.)
    assert backward(**bad) == INVALID


def test_nothing_to_do():
    assert forward(M=0, z=None, g=None, u=None) == 0
    assert forward(N=0, z=None, g=None, u=None) == 0
    assert backward(dx=None, dwg=None, dwu=None) == 0
    assert backward(M=0, dx=None, dwg=None, dwu=None) == 0


def test_tile_refusals():
    set_tile = mg.load().mgemm_set_gated_tile
    handle = ctypes.create_string_buffer(4096)
    h = ctypes.addressof(handle)
    assert set_tile(None, 0, 128, 1) == INVALID
    for bad in ((-1, 128, 1), (3, 128, 1), (0, 64, 1), (0, 192, 0), (0, 128, -1), (0, 128, 33)):
        assert set_tile(h, *bad) == INVALID
    assert set_tile(h, 2, 256, 32) == 0 and set_tile(h, 2, 0, 0) == 0
