"""Z = SiLU(G) U of gates far below zero on the GPU against the formula in 64
bits: SiLU(G) is subnormal in FP32 below -91 and 0 below -108, and U brings the
product back into range.  The 16-bit block and the 4-bit gated pair."""
import numpy as np
import pytest
import torch

import dense_gemm_mgemm_amd as mg
from oracle import gated, mx4
from test_gated_gpu import EPS as EPS16, TINY, Block, h, rounded, say  # noqa: F401
from test_mx4_gpu import EPS, TORCH, quantize

pytestmark = pytest.mark.gpu

# Sums of a few powers of two times 1 to 1.5: exact in E2M1 blocks and in BF16.
FAR = np.array([-48.0, -64.0, -80.0, -88.0, -92.0, -96.0, -104.0, -112.0, -128.0, -144.0])
BIG = 2.0 ** np.array([0.0, 20.0, 30.0, 60.0, 100.0, 100.0, 90.0, 100.0, 100.0, 120.0])


@pytest.mark.parametrize("size,ksplit", [(0, 0), (128, 2), (256, 1), (256, 2)])
def test_forward(h, size, ksplit):  # noqa: F811
    """Z within its rounding to BF16 and 4e-6 of SiLU's FP32 arithmetic, with no absolute slack."""
    say("gated_forward far gates", size, ksplit)
    n, K = len(FAR), 128
    x, wg, wu = np.zeros((n, K)), np.zeros((K, n)), np.zeros((K, n))
    x[:, :n] = np.eye(n)
    wg[:n], wu[:n] = rounded(FAR[:, None] * np.ones(n), "bf16"), rounded(BIG[:, None] * np.linspace(1, 1.9, n), "bf16")
    b = Block(h, "row", n, n, K, "bf16", x, wg, wu)
    try:
        mg.mgemm_set_gated_tile(h, 0, size, ksplit)
        z, _, _ = b.forward()
        torch.cuda.synchronize()
    finally:
        mg.mgemm_set_gated_tile(h, 0)
    zo = gated.forward(x, wg, wu)[0]
    assert np.abs(zo).max() < 2.0 ** 127
    off = np.abs(z.double().cpu().numpy() - zo) > (EPS16["bf16"] + 4e-6) * np.abs(zo) + TINY["bf16"]
    assert not off.any(), [(FAR[i], z[i, j].item(), zo[i, j]) for i, j in np.argwhere(off)[:4]]


# Decode kernel quantising itself and from codes, tiles, and the scalar kernel (weights of odd strides).
@pytest.mark.parametrize("M,K,pad", [(4, 320, 0), (16, 4096, 0), (300, 320, 0), (40, 320, 1)])
@pytest.mark.parametrize("ztype", ["f32", "bf16"])
def test_gated_pair(h, M, K, pad, ztype):  # noqa: F811
    """The same of the 4-bit pair: one value in each block of a weight's row, which E2M1 and a power of two hold."""
    say("gated_mx4 far gates", M, K, pad, ztype)
    n, nb = len(FAR), K // 32
    x = torch.zeros(M, K, device="cuda")
    x[:, 0] = 1.0
    w = torch.zeros(2, n, K, device="cuda", dtype=torch.float64)
    # -48 .. -144 over up to three blocks of a row, each 4 or 6 times a power of two.
    left = FAR.copy()
    for i in range(3):
        step = np.array([max((v for e in range(9) for v in (2.0 ** e, 1.5 * 2.0 ** e) if v <= -f), default=0.0)
                         for f in left])
        w[0, :, 32 * i] = torch.from_numpy(-step).cuda()
        left = left + step
        x[:, 32 * i] = 1.0
    assert not left.any()
    w[1, :, 0] = torch.from_numpy(BIG * 1.5).cuda()
    q, s = [], []
    for i in range(2):
        a, b = quantize(h, w[i].float(), 16 * nb, -(-nb // 16) * 16)
        wide = torch.zeros(n, 16 * nb + pad, dtype=torch.uint8, device="cuda")
        wide[:, :16 * nb] = a
        q.append(wide)
        s.append(b)
    z = torch.full((M, n), float("nan"), dtype=TORCH[ztype], device="cuda")
    mg.mgemm_gated_mx4(h, M, n, K, x, K, "f32", q[0], s[0], q[1], s[1], 16 * nb + pad, s[0].stride(0), z, n, ztype)
    torch.cuda.synchronize()
    g, u = FAR, BIG * 1.5
    zo = mx4.silu(g) * u
    assert np.abs(zo).max() < 2.0 ** 127 and np.abs(zo).min() > 2.0 ** -126
    got = z.double().cpu().numpy()
    off = np.abs(got - zo) > (EPS[ztype] + 4e-6) * np.abs(zo)
    assert not off.any(), [(FAR[j], got[i, j], zo[j]) for i, j in np.argwhere(off)[:4]]
