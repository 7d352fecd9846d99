"""4-bit products at the ends of their format and in every form on the GPU,
against the oracle (oracle/mx4.py): all scale bytes in every kernel."""
import numpy as np
import pytest
import torch

import dense_gemm_mgemm_amd as mg  # noqa: F401
from oracle import mx4
from test_mx4_gpu import TILES, codes, h, product, say  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
@pytest.mark.parametrize("kernel", ["mx4_general", "mx4_skinny"] + TILES)
def test_every_scale_byte(h, kernel, shift):  # noqa: F811
    """Scale bytes 0 to 254 against one another.  The first block of a row holds its values, the others zero codes under
    any scale, so an output is one block's sum times 2^(sa + sb - 254): exact in FP32 where the products of its range
    are normal numbers, within one flush of each of its 32 products below, and not looked at where it overflows."""
    M, N, K = 64, 255, 32 * 6
    say("run_mx4 scale bytes", kernel, shift)
    rng = np.random.default_rng(shift)
    nb = K // 32
    a, b = codes(rng, M, K, 16 * nb, 16, 0, 255), codes(rng, N, K, 16 * nb, 16, 0, 255)
    for x in (a, b):
        x[0][:, 16:] = 0
        x[0][5] = 0                                   # a row of zeros only
    a[1][:, 0] = torch.arange(M, device="cuda").mul(4).add(shift).clamp(max=254).to(torch.uint8)
    b[1][:, 0] = torch.arange(N, device="cuda").to(torch.uint8)
    av, bv = (mx4.decode(x[0].cpu().numpy(), x[1].cpu().numpy()[:, :nb], K) for x in (a, b))
    want, mag = av @ bv.T, np.abs(av) @ np.abs(bv).T
    e = a[1][:, :1].cpu().numpy().astype(int) + b[1][:, 0].cpu().numpy().astype(int) - 254
    c = product(h, kernel, M, N, K, a, b).cpu().double().numpy()
    held = mag < 2.0 ** 127
    normal = held & (e - 2 >= -126)                   # the least product of two codes is 1/4
    assert normal.sum() > 0.4 * M * N and (e[normal] > 100).any() and (e[normal] < -100).any()
    assert np.array_equal(c[normal], want[normal]), np.argwhere(normal & (c != want))[:5]
    low = held & ~normal
    assert (np.abs(c - want)[low] <= 33 * 2.0 ** -126).all()
    assert (c[5] == 0).all() and (c[:, 5] == 0).all()
