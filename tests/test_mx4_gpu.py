"""Microscaled 4-bit path on the GPU against its oracle (oracle/mx4.py):
quantisation bit for bit, products bit for bit where FP32 sums are exact and
within the derived bound otherwise, edges, strides, splits and streams."""
import sys

import numpy as np
import pytest
import torch

import dense_gemm_mgemm_amd as mg
from oracle import mx4

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = {t: torch.finfo(d).eps / 2 for t, d in TORCH.items()}
TILES = ["mx4_mfma_256x256", "mx4_mfma_256x192", "mx4_mfma_128x192", "mx4_mfma_64x192"]


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.load()
    handle = mg.mgemm_create()
    yield handle
    mg.mgemm_destroy(handle)


def up(n, m):
    return -(-n // m) * m


def special(K):
    """Rows that hold what rounding and scaling can get wrong."""
    v = mx4.VALUES
    mids = (v[:-1] + v[1:]) / 2
    pool = np.concatenate([v, -v, mids, -mids, np.nextafter(mids.astype(np.float32), np.float32(9)).astype(float),
                           np.nextafter(mids.astype(np.float32), np.float32(0)).astype(float), [7.5, -7.75]])
    rows = []
    for e in (0, 1, -3, 20, -30, 100, -124, -126):
        r = np.resize(pool, K) * 2.0 ** e
        r[0] = 6.0 * 2.0 ** e
        rows.append(r)
    z = np.zeros(K)
    z[::3] = -0.0
    rows += [z, np.full(K, 2.0 ** -149), np.full(K, -3e38)]
    for bad in (np.nan, np.inf, -np.inf):
        r = np.resize(pool, K).copy()
        r[K // 2] = bad
        rows.append(r)
    return np.array(rows)


def quantize(h, x, ldq, lds):
    M, K = x.shape
    q = torch.full((M, ldq), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((M, lds), 0xA5, dtype=torch.uint8, device="cuda")
    dt = {v: k for k, v in TORCH.items()}[x.dtype]
    mg.mgemm_quantize_mx4(h, M, K, x, x.stride(0), dt, q, ldq, s, lds)
    torch.cuda.synchronize()
    return q, s


@pytest.mark.parametrize("xtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K,pad,qpad,spad", [(3, 1, 0, 0, 0), (37, 300, 4, 0, 3), (16, 4096, 0, 0, 0),
                                               (129, 95, 1, 1, 5), (7, 8200, 8, 16, 7), (5000, 33, 7, 4, 1)])
def test_quantize_and_back(h, xtype, M, K, pad, qpad, spad):
    say("quantize_mx4", xtype, M, K, pad)
    rng = np.random.default_rng(M + K)
    x = rng.standard_normal((M, K)) * np.exp(rng.uniform(-8, 8, (M, 1)))
    x = np.concatenate([x, special(K)])
    wide = torch.full((x.shape[0], K + pad), float("nan"), dtype=TORCH[xtype])
    wide[:, :K] = torch.from_numpy(x).to(TORCH[xtype])
    xv = wide[:, :K].double().numpy()
    nb = -(-K // 32)
    q, s = quantize(h, wide.cuda()[:, :K], 16 * nb + qpad, nb + spad)
    qo, so = mx4.quantize(xv)
    qc, sc = q.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(sc[:, :nb], so), np.argwhere(sc[:, :nb] != so)[:5]
    assert np.array_equal(qc[:, :16 * nb], qo), np.argwhere(qc[:, :16 * nb] != qo)[:5]
    assert (qc[:, 16 * nb:] == 0xA5).all() and (sc[:, nb:] == 0xA5).all()
    want = torch.from_numpy(mx4.decode(qo, so, K))
    for ytype in ("f32", xtype):
        y = torch.full((x.shape[0], K + pad), 77.0, dtype=TORCH[ytype], device="cuda")
        mg.mgemm_dequantize_mx4(h, x.shape[0], K, q, q.stride(0), s, s.stride(0), y, K + pad, ytype)
        torch.cuda.synchronize()
        assert (y[:, K:] == 77.0).all()
        got, ref = y[:, :K].cpu(), want.to(TORCH[ytype])
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(ref)), ytype


def codes(rng, rows, K, ldq, lds, lo=126, hi=129):
    """Random codes and scales on the GPU (padding poisoned) and their values."""
    nb = -(-K // 32)
    c = rng.integers(0, 16, (rows, nb * 32), dtype=np.uint8)
    c[:, K:] = 0
    packed = c[:, 0::2] | (c[:, 1::2] << 4)
    q = np.full((rows, ldq), 0xFF, np.uint8)
    q[:, :16 * nb] = packed
    s = np.full((rows, lds), 0xFF, np.uint8)
    s[:, :nb] = rng.integers(lo, hi, (rows, nb), dtype=np.uint8)
    return torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), mx4.decode(packed, s[:, :nb], K)


def product(h, kernel, M, N, K, a, b, ctype="f32", alpha=1.0, beta=0.0, c0=None, ldc=None, ksplit=0, stream=None):
    ldc = ldc or N
    c = torch.full((M, ldc), float("nan"), dtype=TORCH[ctype], device="cuda") if c0 is None else c0.clone()
    mg.mgemm_run_mx4(h, kernel, M, N, K, alpha, a[0], a[0].stride(0), a[1], a[1].stride(0), b[0], b[0].stride(0),
                     b[1], b[1].stride(0), beta, c, ldc, ctype, ksplit=ksplit, stream=stream)
    torch.cuda.synchronize()
    return c


SIZES = [(1, 1, 1), (5, 17, 31), (64, 96, 128), (33, 200, 160), (17, 70, 511), (64, 193, 1030), (256, 256, 512),
         (300, 260, 700), (130, 400, 2081), (257, 193, 4096), (513, 776, 320)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("kernel", ["auto", "mx4_general", "mx4_skinny"] + TILES)
def test_product_bit_exact(h, kernel, M, N, K):
    # Codes are multiples of 1/2 up to 6 and scales 1/2, 1 or 2: every product is a multiple of 2^-4 up to 144, so
    # sums of up to 4096 stay below 2^24 multiples of 2^-4 and FP32 sums in any order are exact.
    if kernel == "mx4_skinny" and M > 64:
        pytest.skip("at most 64 rows")
    say("run_mx4", kernel, M, N, K)
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    nb = -(-K // 32)
    a = codes(rng, M, K, 16 * nb, up(nb, 16))
    b = codes(rng, N, K, 16 * nb + 16, up(nb, 16) + 16)
    want = a[2] @ b[2].T
    c = product(h, kernel, M, N, K, a, b)
    assert np.array_equal(c.cpu().double().numpy(), want)
    # alpha, beta, a wider C whose padding stays, each type rounded once.
    c0 = torch.from_numpy(rng.integers(-8, 9, (M, N + 5)).astype(np.float32)).cuda()
    for ctype in ("f32", "f16", "bf16"):
        c = product(h, kernel, M, N, K, a, b, ctype, -0.5, 2.0, c0.to(TORCH[ctype]), N + 5)
        ref = torch.from_numpy(-0.5 * want + 2.0 * c0[:, :N].cpu().double().numpy()).to(TORCH[ctype])
        assert torch.equal(c[:, :N].cpu(), ref), ctype
        assert torch.equal(c[:, N:], c0.to(TORCH[ctype])[:, N:])


@pytest.mark.parametrize("kernel", TILES)
@pytest.mark.parametrize("ksplit", [2, 3, 7, 32])
def test_product_split(h, kernel, ksplit):
    for M, N, K in ((70, 200, 1900), (300, 270, 4000)):
        say("run_mx4 split", kernel, ksplit, M, N, K)
        rng = np.random.default_rng(K)
        nb = -(-K // 32)
        a, b = codes(rng, M, K, 16 * nb, up(nb, 16)), codes(rng, N, K, 16 * nb, up(nb, 16))
        c = product(h, kernel, M, N, K, a, b, "f16", 0.25, 0.0, ksplit=ksplit)
        assert torch.equal(c.cpu(), torch.from_numpy(0.25 * (a[2] @ b[2].T)).to(torch.float16))


def test_unaligned_operands_take_the_scalar_kernel(h):
    # Odd strides and bases: any alignment gives the same bits.
    M, N, K = 70, 65, 333
    rng = np.random.default_rng(1)
    nb = -(-K // 32)
    a, b = codes(rng, M, K, 16 * nb + 1, nb + 2), codes(rng, N, K, 16 * nb + 3, nb)
    assert np.array_equal(product(h, "auto", M, N, K, a, b).cpu().double().numpy(), a[2] @ b[2].T)


@pytest.mark.parametrize("kernel", ["mx4_general", "mx4_skinny"] + TILES)
def test_scales_of_every_size_and_nan(h, kernel):
    # One block per product: 2^(sa + sb - 254) from 2^-100 to 2^100 is exact; byte 255 poisons its row and column only.
    M, N, K = 40, 50, 32 * 9 if kernel == "mx4_general" else 32 * 6
    rng = np.random.default_rng(2)
    nb = K // 32
    a, b = codes(rng, M, K, 16 * nb, 16), codes(rng, N, K, 16 * nb, 16)
    for q, s, _ in (a, b):
        q[:, 16:16 * nb] = 0                          # only the first block of a row holds values
        s[:, 0] = torch.from_numpy(rng.integers(77, 178, q.shape[0]).astype(np.uint8)).cuda()
    av, bv = (mx4.decode(x[0].cpu().numpy()[:, :16 * nb], x[1].cpu().numpy()[:, :nb], K) for x in (a, b))
    want = av @ bv.T
    c = product(h, kernel, M, N, K, a, b).cpu().double().numpy()
    assert np.array_equal(c, want)
    a[1][3, nb - 1], b[1][11, 2] = 255, 255
    c = product(h, kernel, M, N, K, a, b).cpu().double().numpy()
    nan = np.isnan(c)
    assert nan[3].all() and nan[:, 11].all()
    nan[3], nan[:, 11] = False, False
    assert not nan.any()
    keep = np.ones_like(want, bool)
    keep[3], keep[:, 11] = False, False
    assert np.array_equal(c[keep], want[keep])


def weights(h, rng, N, K):
    w = torch.from_numpy((rng.standard_normal((N, K)) / np.sqrt(K)).astype(np.float32)).cuda()
    nb = -(-K // 32)
    q, s = quantize(h, w, 16 * nb, up(nb, 16))
    s[:, nb:] = 0xFF
    return q, s, mx4.decode(q.cpu().numpy(), s.cpu().numpy()[:, :nb], K)


def bound(y, mag, K, t):
    """One rounding to t, and FP32 sums of K products of magnitude sum `mag` (each addition off by half a step)."""
    return EPS[t] * np.abs(y) + (K + 2) * 2.0 ** -24 * mag + 2.0 ** -24


@pytest.mark.parametrize("M,N,K", [(1, 1, 33), (1, 5000, 1000), (3, 100, 4096), (4, 12300, 64), (5, 48, 2000),
                                   (16, 333, 1504), (17, 64, 96), (48, 1000, 300), (65, 130, 1000), (700, 500, 160)])
@pytest.mark.parametrize("xtype,pad", [("bf16", 0), ("bf16", 3), ("f16", 8), ("f32", 4), ("f32", 0)])
def test_linear_and_gated(h, M, N, K, xtype, pad):
    say("linear_mx4", M, N, K, xtype, pad)
    rng = np.random.default_rng(M + N + K)
    x = torch.full((M, K + pad), float("nan"))
    x[:, :K] = torch.from_numpy(rng.standard_normal((M, K)) * (1 + 7 * (rng.random(K) < 0.02)))
    x = x.to(TORCH[xtype]).cuda()[:, :K]
    xq = mx4.decode(*mx4.quantize(x.cpu().double().numpy()), K)
    wg, wu = weights(h, rng, N, K), weights(h, rng, N, K)
    g, u = xq @ wg[2].T, xq @ wu[2].T
    mg_, mu = np.abs(xq) @ np.abs(wg[2]).T, np.abs(xq) @ np.abs(wu[2]).T
    for yt in ("f32", xtype):
        y = torch.full((M, N + 3), 55.0, dtype=TORCH[yt], device="cuda")
        mg.mgemm_linear_mx4(h, M, N, K, x, x.stride(0), xtype, wg[0], wg[0].stride(0), wg[1], wg[1].stride(0), y,
                            N + 3, yt)
        torch.cuda.synchronize()
        assert (y[:, N:] == 55.0).all()
        err = np.abs(y[:, :N].cpu().double().numpy() - g)
        assert (err <= bound(g, mg_, K, yt)).all(), (yt, err.max())
        z = torch.full((M, N + 3), 55.0, dtype=TORCH[yt], device="cuda")
        mg.mgemm_gated_mx4(h, M, N, K, x, x.stride(0), xtype, wg[0], wg[1], wu[0], wu[1], wg[0].stride(0),
                           wg[1].stride(0), z, N + 3, yt)
        torch.cuda.synchronize()
        assert (z[:, N:] == 55.0).all()
        want = mx4.silu(g) * u
        # The sums' errors through SiLU (slope at most 1.1) and the product; SiLU itself within 4e-6 relative.
        dg, du = (K + 2) * 2.0 ** -24 * mg_, (K + 2) * 2.0 ** -24 * mu
        lim = EPS[yt] * np.abs(want) + 1.1 * dg * (np.abs(u) + du) + np.abs(mx4.silu(g)) * du + 4e-6 * np.abs(want)
        err = np.abs(z[:, :N].cpu().double().numpy() - want)
        assert (err <= lim + 2.0 ** -24).all(), (yt, err.max())


def test_rows_in_bands(h):
    # 40000 rows of 5000 values are 107 MB of codes and scales: two bands through the workspace.
    M, N, K = 40000, 70, 5000
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-2, 3, (M, K), generator=gen, device="cuda").to(torch.bfloat16)
    x[:, ::32] = 4                                    # every block's largest value: scale 1, exact codes
    w = torch.randint(-2, 3, (N, K), generator=gen, device="cuda").float()
    w[:, ::32] = 4
    q, s = quantize(h, w, 16 * 157, 160)
    y = torch.empty(M, N, dtype=torch.float32, device="cuda")
    mg.mgemm_linear_mx4(h, M, N, K, x, K, "bf16", q, 16 * 157, s, 160, y, N, "f32")
    torch.cuda.synchronize()
    # Integers: exact in FP32 whatever the order.
    assert torch.equal(y, x.float() @ w.t())


def test_empty_sizes(h):
    c = torch.full((3, 4), 2.0, device="cuda")
    b = torch.zeros(64, dtype=torch.uint8, device="cuda")
    mg.mgemm_run_mx4(h, "auto", 3, 4, 0, 1.0, None, 1, None, 1, None, 1, None, 1, 0.5, c, 4, "f32")
    torch.cuda.synchronize()
    assert (c == 1.0).all()
    mg.mgemm_linear_mx4(h, 3, 4, 0, None, 1, "f32", None, 1, None, 1, c, 4, "f32")
    torch.cuda.synchronize()
    assert (c == 0.0).all()
    mg.mgemm_linear_mx4(h, 0, 4, 32, None, 32, "f32", b, 16, b, 1, None, 4, "f32")
    mg.mgemm_gated_mx4(h, 3, 0, 32, c, 32, "f32", b, b, b, b, 16, 1, None, 1, "f32")
    torch.cuda.synchronize()


def test_other_stream_and_graph(h):
    # Calls on a stream that is not the current one, and replays of a captured call, against the eager result.
    rng = np.random.default_rng(9)
    N, K = 300, 1000
    w = weights(h, rng, N, K)
    side = torch.cuda.Stream()
    for M in (3, 40, 200):
        x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).cuda()
        y, z = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")

        def call(out, stream=None):
            mg.mgemm_linear_mx4(h, M, N, K, x, K, "f32", w[0], w[0].stride(0), w[1], w[1].stride(0), out, N, "f32",
                                stream=stream)
        call(y)
        torch.cuda.synchronize()
        call(z, side)
        side.synchronize()
        assert torch.equal(y, z)
        g = torch.cuda.CUDAGraph()
        z.zero_()
        with torch.cuda.graph(g):
            call(z)
        for i in range(3):
            x.mul_(-1.0)
            call(y)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, z), (M, i)


@pytest.mark.parametrize("M,N,K", [(1, 50, 700), (20, 70, 1500), (64, 33, 250)])
def test_scale_rows_of_eight_bytes(h, M, N, K):
    # Scale strides that are multiples of 8 and not of 16: the decode kernel, whose last load ends with the row.
    rng = np.random.default_rng(K)
    nb = -(-K // 32)
    lds = up(nb, 8) + (8 if up(nb, 8) % 16 == 0 else 0)
    a, b = codes(rng, M, K, 16 * nb, lds), codes(rng, N, K, 16 * nb, lds)
    for kernel in ("auto", "mx4_skinny"):
        say("run_mx4 scale stride", lds, kernel, M, N, K)
        assert np.array_equal(product(h, kernel, M, N, K, a, b).cpu().double().numpy(), a[2] @ b[2].T)
