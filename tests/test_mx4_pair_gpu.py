"""Every kernel and split of the 4-bit products that quantise their activations
(mgemm_linear_mx4, mgemm_gated_mx4) on the GPU, on values whose codes and sums
are exact; sizes whose time model takes each form of the gated pair; row bands;
offsets past 31 bits."""
import numpy as np
import pytest
import torch

import dense_gemm_mgemm_amd as mg
from oracle import mx4
from test_mx4_gpu import EPS, TILES, TORCH, codes, h, product, quantize, say, up  # noqa: F401

pytestmark = pytest.mark.gpu

PAIR_TILES = ["mx4_mfma_256x192", "mx4_mfma_128x192"]
KERNELS = [("auto", 0), ("mx4_general", 1), ("mx4_skinny", 1)] + [(k, s) for k in TILES for s in (1, 2, 3, 7, 32)]


def integers(gen, rows, K):
    """Values that E2M1 with scale 1 holds: integers up to 2, each block's largest 4."""
    x = torch.randint(-2, 3, (rows, K), generator=gen, device="cuda").float()
    x[:, ::32] = 4
    return x


def gate_error(z, g, u, ztype):
    """Whether Z of exact sums is off by more than its rounding and 4e-6 of SiLU's FP32 arithmetic."""
    zo = g * torch.sigmoid(g) * u
    err = (z.double() - zo).abs()
    return (err > (EPS[ztype] + 4e-6) * zo.abs() + 2.0 ** -25).any().item()


def forced(h, kernel, ksplit, call):  # noqa: F811
    try:
        mg.mgemm_set_mx4_kernel(h, kernel, ksplit)
        call()
        torch.cuda.synchronize()
    finally:
        mg.mgemm_set_mx4_kernel(h)


@pytest.mark.parametrize("M,N,K", [(1, 7, 33), (16, 97, 1000), (20, 200, 1900), (50, 96, 4000), (64, 193, 130),
                                   (130, 300, 1030), (300, 270, 1900)])
@pytest.mark.parametrize("kernel,ksplit", KERNELS)
def test_every_kernel(h, M, N, K, kernel, ksplit):  # noqa: F811
    if kernel == "mx4_skinny" and M > 64:
        return                                        # refused: tests of refusals
    say("mx4 forced", kernel, ksplit, M, N, K)
    rng = np.random.default_rng(M + N + K)
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    nb = -(-K // 32)
    x = integers(gen, M, K)
    # Weights up to 6 in blocks worth 1/8 to 1/2: sums of quarters of 1/8, exact in FP32.
    wg, wu = (codes(rng, N, K, 16 * nb + 16, up(nb, 16), 124, 127) for _ in range(2))
    g, u = (x.double() @ torch.from_numpy(w[2]).cuda().t() for w in (wg, wu))
    for t in ("f32", "f16", "bf16"):
        y = torch.full((M, N + 3), 55.0, dtype=TORCH[t], device="cuda")
        forced(h, kernel, ksplit, lambda: mg.mgemm_linear_mx4(
            h, M, N, K, x, K, "f32", wg[0], wg[0].stride(0), wg[1], wg[1].stride(0), y, N + 3, t))
        assert (y[:, N:] == 55.0).all() and torch.equal(y[:, :N], g.to(TORCH[t])), t
        if kernel in TILES and kernel not in PAIR_TILES:
            continue
        z = torch.full((M, N + 3), 55.0, dtype=TORCH[t], device="cuda")
        forced(h, kernel, ksplit, lambda: mg.mgemm_gated_mx4(
            h, M, N, K, x, K, "f32", wg[0], wg[1], wu[0], wu[1], wg[0].stride(0), wg[1].stride(0), z, N + 3, t))
        zo = g * torch.sigmoid(g) * u
        held = zo.abs() < torch.finfo(TORCH[t]).max * (1 - 2 * EPS[t])
        assert (z[:, N:] == 55.0).all()
        assert not gate_error(torch.where(held, z[:, :N].double(), 0.0), torch.where(held, g, 0.0), u, t), t


# Sizes that the time model gives to the decode kernel's wider blocks, split tiles and the 256-row tile.
@pytest.mark.parametrize("M,N,K", [(32, 4096, 4096), (31, 4000, 4000), (64, 1536, 4096), (61, 1500, 4090),
                                   (128, 4096, 4096), (117, 4100, 4000), (1024, 1536, 4096), (1000, 1541, 4099),
                                   (1024, 12288, 4096), (3000, 2000, 1000)])
def test_pair_of_model_sizes(h, M, N, K):  # noqa: F811
    say("gated_mx4 model sizes", M, N, K)
    gen = torch.Generator(device="cuda").manual_seed(M)
    x, wg, wu = integers(gen, M, K), integers(gen, N, K), integers(gen, N, K)
    nb = -(-K // 32)
    (qg, sg), (qu, su) = (quantize(h, w, 16 * nb, up(nb, 16)) for w in (wg, wu))
    z = torch.empty(M, N, device="cuda")
    mg.mgemm_gated_mx4(h, M, N, K, x, K, "f32", qg, sg, qu, su, qg.stride(0), sg.stride(0), z, N, "f32")
    torch.cuda.synchronize()
    assert not gate_error(z, (x @ wg.t()).double(), (x @ wu.t()).double(), "f32")


def test_pair_with_odd_strides(h):  # noqa: F811
    M, N, K = 70, 65, 333
    say("gated_mx4 odd strides")
    rng = np.random.default_rng(1)
    gen = torch.Generator(device="cuda").manual_seed(1)
    nb = -(-K // 32)
    x = integers(gen, M, K)
    wg, wu = (codes(rng, N, K, 16 * nb + 3, nb, 124, 127) for _ in range(2))
    z = torch.empty(M, N, device="cuda")
    mg.mgemm_gated_mx4(h, M, N, K, x, K, "f32", wg[0], wg[1], wu[0], wu[1], 16 * nb + 3, nb, z, N, "f32")
    torch.cuda.synchronize()
    assert not gate_error(z, *(x.double() @ torch.from_numpy(w[2]).cuda().t() for w in (wg, wu)), "f32")


def test_pair_in_bands(h):  # noqa: F811
    M, N, K = 40000, 70, 5000                         # 107 MB of codes and scales: two bands
    say("gated_mx4 bands")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, wg, wu = integers(gen, M, K), integers(gen, N, K), integers(gen, N, K)
    (qg, sg), (qu, su) = (quantize(h, w, 16 * 157, 160) for w in (wg, wu))
    z = torch.empty(M, N, device="cuda")
    mg.mgemm_gated_mx4(h, M, N, K, x, K, "f32", qg, sg, qu, su, 16 * 157, 160, z, N, "f32")
    torch.cuda.synchronize()
    assert not gate_error(z, (x @ wg.t()).double(), (x @ wu.t()).double(), "f32")


def test_nan_in_every_kernel(h):  # noqa: F811
    """A NaN or an infinity in a row of X makes that row of Y and Z NaN and no other."""
    M, N, K = 40, 70, 700
    gen = torch.Generator(device="cuda").manual_seed(3)
    nb = -(-K // 32)
    x, wg = integers(gen, M, K), integers(gen, N, K)
    x[7, 300], x[33, 699] = float("nan"), float("-inf")
    q, s = quantize(h, wg, 16 * nb, up(nb, 16))
    good = torch.ones(M, dtype=torch.bool, device="cuda")
    good[7] = good[33] = False
    g = x[good] @ wg.t()
    for kernel, ksplit in KERNELS:
        say("mx4 NaN", kernel, ksplit)
        y = torch.empty(M, N, device="cuda")
        forced(h, kernel, ksplit, lambda: mg.mgemm_linear_mx4(h, M, N, K, x, K, "f32", q, 16 * nb, s, s.stride(0), y,
                                                              N, "f32"))
        assert torch.isnan(y[~good]).all() and torch.equal(y[good], g)


def test_offsets_past_31_bits(h):  # noqa: F811
    """70000 rows of 66016 values: 4.6e9 elements, 2.3e9 bytes of codes; as activations, as weights, and 66000 x 33000
    outputs."""
    M, K, N = 70000, 66016, 48
    say("mx4 large: quantise")
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    for m in range(0, M, 10000):
        x[m:m + 10000] = torch.randint(-2, 3, (min(10000, M - m), K), generator=gen, device="cuda", dtype=torch.int8)
    x[:, ::32] = 4
    nb = K // 32
    q, s = quantize(h, x, 16 * nb, up(nb, 16))
    back = torch.empty_like(x)
    mg.mgemm_dequantize_mx4(h, M, K, q, 16 * nb, s, s.stride(0), back, K, "bf16")
    torch.cuda.synchronize()
    assert torch.equal(back, x)
    del back
    w = integers(gen, N, K)
    wq, ws = quantize(h, w, 16 * nb, up(nb, 16))
    # Sums of 66016 products of up to 16: below 2^24, exact in FP32.
    want = torch.cat([x[m:m + 10000].float() @ w.t() for m in range(0, M, 10000)])
    for kernel in ["mx4_general"] + TILES:
        say("mx4 large: activations", kernel)
        assert torch.equal(product(h, kernel, M, N, K, (q, s), (wq, ws)), want)
    for kernel in ["mx4_general", "mx4_skinny"] + TILES:
        say("mx4 large: weights", kernel)
        assert torch.equal(product(h, kernel, N, M, K, (wq, ws), (q, s)), want.t())
    del q, s, x, want
    M, N, K = 66000, 33000, 64
    say("mx4 large: outputs")
    x, w = integers(gen, M, K), integers(gen, N, K)
    wq, ws = quantize(h, w, 32, 16)
    y = torch.empty(M, N, device="cuda")
    for kernel in ["auto", "mx4_general"] + TILES:
        say("mx4 large: outputs", kernel)
        y.fill_(float("nan"))
        forced(h, kernel, 0, lambda: mg.mgemm_linear_mx4(h, M, N, K, x, K, "f32", wq, 32, ws, 16, y, N, "f32"))
        for m in range(0, M, 11000):
            assert torch.equal(y[m:m + 11000], x[m:m + 11000] @ w.t())
