"""The microscaled 4-bit oracle against the specification's own statements,
the argument checks of the entry points (no GPU is reached), and the generated
code of their kernels."""
import ctypes
import os
import re

import numpy as np
import pytest

import dense_gemm_mgemm_amd as mg
from oracle import mx4
from tests import test_codegen as cg


def test_codes_round_to_nearest_even():
    # Midpoints of neighbours go to the even code, anything beyond to the nearer one.
    v = mx4.VALUES
    mids = (v[:-1] + v[1:]) / 2
    assert list(mx4.encode(v)) == list(range(8)) and list(mx4.encode(-v)) == list(range(8, 16))
    assert list(mx4.encode(mids)) == [0, 2, 2, 4, 4, 6, 6]
    assert list(mx4.encode(np.nextafter(mids, 9))) == [1, 2, 3, 4, 5, 6, 7]
    assert list(mx4.encode(np.nextafter(mids, 0))) == [0, 1, 2, 3, 4, 5, 6]
    assert list(mx4.encode([7.9, 1e30, -1e30])) == [7, 7, 15]


def test_scale_is_the_largest_binade():
    # amax in [4, 8) 2^e gets scale 2^e: its code is in the top binade {4, 6}.
    for amax, e in ((4.0, 0), (7.99, 0), (8.0, 1), (3.99, -1), (1.0, -2), (2.0 ** -126, -127), (2.0 ** -140, -127)):
        x = np.zeros((1, 40))
        x[0, 33] = amax
        q, s = mx4.quantize(x)
        assert list(s[0]) == [0, 127 + e]
        assert q.shape == (1, 32)


def test_round_trip_of_representable_values():
    rng = np.random.default_rng(0)
    q = rng.integers(0, 256, (5, 48), dtype=np.uint8)
    s = rng.integers(100, 150, (5, 3), dtype=np.uint8)
    q[:, 0::16] |= 0x07                             # a 6 in every block fixes its scale
    v = mx4.decode(q, s, 96)
    q2, s2 = mx4.quantize(v)
    assert np.array_equal(s2, s) and np.array_equal(q2, q)


def test_non_finite_blocks():
    x = np.ones((1, 96))
    x[0, 5], x[0, 40] = np.nan, -np.inf
    q, s = mx4.quantize(x)
    assert list(s[0]) == [255, 255, 125] and not q[0, :32].any()
    assert np.isnan(mx4.decode(q, s, 96)[0, :64]).all() and (mx4.decode(q, s, 96)[0, 64:] == 1).all()


# A zeroed block stands for a handle: the checks that refuse a call come before any use of the device.
KEEP = ctypes.create_string_buffer(4096)
P = ctypes.addressof(KEEP)


def refused(call, status=mg.MGEMM_ERR_INVALID_ARG):
    with pytest.raises(mg.MgemmError) as e:
        call()
    assert e.value.status == status


@pytest.fixture(scope="module")
def handle():
    block = ctypes.create_string_buffer(4096)
    yield ctypes.addressof(block)
    del block


def test_quantize_refusals(handle):
    def q(h=handle, M=4, K=40, X=P, ldx=40, t="bf16", Q=P, ldq=32, S=P, lds=2):
        mg.mgemm_quantize_mx4(h, M, K, X, ldx, t, Q, ldq, S, lds, stream=0)

    def d(h=handle, M=4, K=40, Q=P, ldq=32, S=P, lds=2, Y=P, ldy=40, t="f32"):
        mg.mgemm_dequantize_mx4(h, M, K, Q, ldq, S, lds, Y, ldy, t, stream=0)
    for f in (q, d):
        for bad in (dict(h=None), dict(M=-1), dict(K=-1), dict(ldq=31), dict(lds=1), dict(t=3), dict(Q=None),
                    dict(S=None), dict(M=2 ** 62)):
            refused(lambda: f(**bad))
        f(M=0, X=None) if f is q else f(M=0, Y=None)          # nothing to do
    refused(lambda: q(ldx=39))
    refused(lambda: q(X=None))
    refused(lambda: d(ldy=39))
    refused(lambda: d(Y=None))
    refused(lambda: q(M=1, K=2 ** 34, ldx=2 ** 34, ldq=2 ** 34, lds=2 ** 30), mg.MGEMM_ERR_UNSUPPORTED)


def test_product_refusals(handle):
    def run(h=handle, kernel="auto", M=4, N=4, K=40, A=P, lda=32, SA=P, ldsa=2, B=P, ldb=32, SB=P, ldsb=2, C=P,
            ldc=4, t="f32", ksplit=0):
        mg.mgemm_run_mx4(h, kernel, M, N, K, 1.0, A, lda, SA, ldsa, B, ldb, SB, ldsb, 0.0, C, ldc, t, stream=0,
                         ksplit=ksplit)

    def linear(h=handle, M=4, N=4, K=40, X=P, ldx=40, xt="bf16", B=P, ldb=32, SB=P, ldsb=2, C=P, ldc=4, t="f32"):
        mg.mgemm_linear_mx4(h, M, N, K, X, ldx, xt, B, ldb, SB, ldsb, C, ldc, t, stream=0)

    def gated(h=handle, M=4, N=4, K=40, X=P, ldx=40, xt="bf16", B=P, Bu=P, ldb=32, SB=P, SBu=P, ldsb=2, C=P, ldc=4,
              t="f32"):
        mg.mgemm_gated_mx4(h, M, N, K, X, ldx, xt, B, SB, Bu, SBu, ldb, ldsb, C, ldc, t, stream=0)
    for f in (run, linear, gated):
        for bad in (dict(h=None), dict(M=-1), dict(N=-1), dict(K=-1), dict(ldb=31), dict(ldsb=1), dict(ldc=3),
                    dict(t=7), dict(B=None), dict(SB=None), dict(C=None)):
            refused(lambda: f(**bad))
        f(M=0)
        f(N=0, C=None)
    for bad in (dict(lda=31), dict(ldsa=1), dict(A=None), dict(SA=None), dict(ksplit=-1), dict(ksplit=2),
                dict(kernel="mx4_general", ksplit=33), dict(kernel="f8_general"), dict(kernel="h_dma_256x256")):
        refused(lambda: run(**bad))
    for f in (linear, gated):
        for bad in (dict(ldx=39), dict(X=None), dict(xt=9)):
            refused(lambda: f(**bad))
    refused(lambda: gated(Bu=None))
    refused(lambda: gated(SBu=None))
    # Forced kernels that cannot run the problem: strides of 17 bytes, 65 rows, a split of the scalar kernel.
    for bad in (dict(kernel="mx4_mfma_256x256", lda=33, ldsa=16, ldsb=16), dict(kernel="mx4_mfma_64x192", ldsa=3),
                dict(kernel="mx4_skinny", M=65), dict(kernel="mx4_general", ksplit=2)):
        refused(lambda: run(**bad), mg.MGEMM_ERR_UNSUPPORTED)


@pytest.mark.skipif(not os.path.exists(cg.HIPCC), reason="hipcc not available")
def test_generated_code(tmp_path):
    # As for the other direct-to-LDS kernels: m0 is written by the copies alone, nothing spills.
    for name in ("k_mx4.hip", "k_mx4_skinny.hip", "k_mx4_quant.hip"):
        text, remarks = cg.device_build(name, tmp_path)
        body = [l.strip() for l in text.splitlines()]
        for i, l in enumerate(body):
            if re.search(r"\bm0\b", l) and not l.startswith(";"):
                assert l.startswith("s_mov_b32 m0,") and body[i + 1] == "s_nop 0", l
                assert body[i + 2].startswith("global_load_lds_dwordx4"), l
        assert max(int(x) for x in re.findall(r"VGPRs Spill: (\d+)", remarks)) == 0, name
        assert max(int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", remarks)) == 0, name
        assert not re.search(r"^\s*v_pk_(add|mul|fma)_f32", text, re.M), name
