"""Refusals of the hook that forces the kernel of 4-bit products of values, on
the CPU: nothing is launched."""
import ctypes

import pytest

import dense_gemm_mgemm_amd as mg

P = 1 << 20                                           # an aligned address that nothing reads


@pytest.fixture()
def handle():
    block = ctypes.create_string_buffer(4096)
    yield ctypes.addressof(block)
    del block


def refused(call, status=mg.MGEMM_ERR_INVALID_ARG):
    with pytest.raises(mg.MgemmError) as e:
        call()
    assert e.value.status == status


def test_refusals(handle):
    for bad in ((None, "auto", 0), (handle, "auto", 1), (handle, "mx4_general", -1), (handle, "mx4_skinny", 33),
                (handle, "f8_general", 0), (handle, "h_dma_256x256", 0)):
        refused(lambda: mg.mgemm_set_mx4_kernel(*bad))
    mg.mgemm_set_mx4_kernel(handle, "mx4_mfma_256x192", 32)
    mg.mgemm_set_mx4_kernel(handle)
