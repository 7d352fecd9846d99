"""The gated block's forward and backward pass on the GPU against its oracle
(oracle/gated.py): bit for bit where every step is exact, within the derived
bound otherwise; layouts, strides, tails, splits, streams and graphs."""
import sys

import numpy as np
import pytest
import torch

import dense_gemm_mgemm_amd as mg
from oracle import gated

pytestmark = pytest.mark.gpu

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = {t: torch.finfo(d).eps / 2 for t, d in TORCH.items()}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}        # half the smallest subnormal step
F32 = 2.0 ** -24


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


def wide(v, ld, dtype, shift=0, fill=float("nan")):
    """v on the GPU with row stride ld, poisoned between rows and `shift` elements into its storage."""
    rows, cols = v.shape
    flat = torch.full((shift + rows * ld,), fill, dtype=TORCH[dtype], device="cuda")
    view = flat[shift:].view(rows, ld)[:, :cols]
    view.copy_(torch.as_tensor(v))
    return view


class Block:
    """One block's operands: values in float64, the GPU's copies, and calls."""

    def __init__(self, h, layout, M, N, K, dtype, x, wg, wu, pad=0, shift=0):
        self.h, self.layout, self.M, self.N, self.K, self.dtype, self.pad = h, layout, M, N, K, dtype, pad
        self.x = wide(x, K + pad, dtype, shift)
        stored = [w if layout == "row" else w.T for w in (wg, wu)]
        self.ldw = stored[0].shape[1] + pad
        self.wg, self.wu = (wide(w, self.ldw, dtype, shift) for w in stored)

    def work(self, backward, stored=False):
        n = mg.mgemm_gated_workspace(self.layout, self.M, self.N, self.K, self.x, self.K + self.pad, self.wg, self.wu,
                                     self.ldw, self.dtype, backward, stored)
        # An odd start: the library aligns it itself.
        return torch.full((n + 3,), 0xFF, dtype=torch.uint8, device="cuda")[3:]

    def out(self, rows, cols, fill=7.0):
        return torch.full((rows, cols + self.pad), fill, dtype=TORCH[self.dtype], device="cuda")

    def forward(self, keep=True, stream=None, outs=None):
        w = self.work(False)
        z, g, u = outs or [self.out(self.M, self.N) for _ in range(3)]
        mg.mgemm_gated_forward(self.h, self.layout, self.M, self.N, self.K, self.x, self.K + self.pad, self.wg, self.wu,
                               self.ldw, z, self.N + self.pad, g if keep else None, u if keep else None,
                               self.N + self.pad, self.dtype, w, w.numel(), stream=stream)
        self.kept = w
        return z, g, u

    def backward(self, dz, g=None, u=None, beta=0.0, outs=None, dx=True, dw=True, stream=None):
        w = self.work(True, g is not None)
        rows, cols = (self.K, self.N) if self.layout == "row" else (self.N, self.K)
        if outs is None:
            outs = [self.out(self.M, self.K), self.out(rows, cols, 3.0), self.out(rows, cols, -2.0)]
        mg.mgemm_gated_backward(self.h, self.layout, self.M, self.N, self.K, self.x, self.K + self.pad, self.wg,
                                self.wu, self.ldw, g, u, g.stride(0) if g is not None else self.N, dz, dz.stride(0),
                                outs[0] if dx else None, self.K + self.pad, outs[1] if dw else None,
                                outs[2] if dw else None, cols + self.pad, beta, self.dtype, w, w.numel(),
                                stream=stream)
        self.kept = w
        return outs

    def grads(self, outs):
        """dX, dWg, dWu as K x N float64, after a check that the padding is untouched."""
        rows, cols = (self.K, self.N) if self.layout == "row" else (self.N, self.K)
        for o, c, f in zip(outs, (self.K, cols, cols), (7.0, 3.0, -2.0)):
            assert (o[:, c:] == f).all()
        dx, a, b = outs[0][:, :self.K], outs[1][:, :cols], outs[2][:, :cols]
        return [v.double().cpu().numpy() for v in ((dx, a, b) if self.layout == "row" else (dx, a.T, b.T))]


def rounded(v, dtype):
    return torch.as_tensor(v).to(TORCH[dtype]).double().numpy()


def ints(rng, shape, top):
    return rng.integers(-top, top + 1, shape).astype(np.float64)


SIZES = [(1, 1, 1), (1, 96, 64), (2, 7, 33), (3, 200, 31), (31, 97, 40), (64, 193, 100), (129, 130, 257), (257, 96, 512),
         (300, 520, 96), (33, 1000, 1001), (640, 40, 65)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("dtype,pad,shift", [("bf16", 0, 0), ("f16", 8, 0), ("bf16", 3, 1), ("f16", 0, 4)])
def test_forward(h, layout, M, N, K, dtype, pad, shift):
    say("gated_forward", layout, M, N, K, dtype, pad, shift)
    rng = np.random.default_rng(M + 3 * N + 5 * K)
    # Integers up to 2 and 3: FP32 sums are exact in any order, so G and U are their values rounded once.
    x, wg, wu = ints(rng, (M, K), 2), ints(rng, (K, N), 3), ints(rng, (K, N), 3)
    b = Block(h, layout, M, N, K, dtype, x, wg, wu, pad, shift)
    z, g, u = b.forward()
    torch.cuda.synchronize()
    for t in (z, g, u):
        assert (t[:, N:] == 7.0).all()
    zo, go, uo = gated.forward(x, wg, wu)
    assert np.array_equal(g[:, :N].double().cpu().numpy(), rounded(go, dtype))
    assert np.array_equal(u[:, :N].double().cpu().numpy(), rounded(uo, dtype))
    # Z: one rounding, SiLU within 4e-6 relative (one FP32 operation after another from exact sums).
    got = z[:, :N].double().cpu().numpy()
    top = float(torch.finfo(TORCH[dtype]).max)
    near = np.abs(zo) < top * (1 - 2 * EPS[dtype])
    assert (np.abs(got - zo)[near] <= ((EPS[dtype] + 4e-6) * np.abs(zo) + TINY[dtype])[near]).all()
    assert (np.abs(got[~near]) >= top * (1 - 4 * EPS[dtype])).all()
    alone, _, _ = b.forward(keep=False)
    torch.cuda.synchronize()
    assert torch.equal(alone, z)


def bound(y, mag, terms, t):
    """One rounding to t, and an FP32 sum of `terms` products whose magnitudes add up to mag."""
    return EPS[t] * np.abs(y) + (terms + 2) * F32 * mag + TINY[t]


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_forward_random(h, layout, dtype):
    M, N, K = 200, 310, 777
    rng = np.random.default_rng(4)
    x, wg, wu = (rounded(v, dtype) for v in (rng.standard_normal((M, K)), rng.standard_normal((K, N)) / 9,
                                             rng.standard_normal((K, N)) / 9))
    z, g, u = (v[:, :N].double().cpu().numpy() for v in Block(h, layout, M, N, K, dtype, x, wg, wu).forward())
    zo, go, uo = gated.forward(x, wg, wu)
    mg_, mu = np.abs(x) @ np.abs(wg), np.abs(x) @ np.abs(wu)
    assert (np.abs(g - go) <= bound(go, mg_, K, dtype)).all()
    assert (np.abs(u - uo) <= bound(uo, mu, K, dtype)).all()
    # The sums' errors through SiLU (slope at most 1.1) and the product.
    dg, du = (K + 2) * F32 * mg_, (K + 2) * F32 * mu
    lim = (EPS[dtype] + 4e-6) * np.abs(zo) + 1.1 * dg * (np.abs(uo) + du) + np.abs(go) * du + TINY[dtype]
    assert (np.abs(z - zo) <= lim).all()


def exact_case(rng, M, N, K):
    """Integers for which every step of the backward pass is exact: G is 0 (s = 1/2, so dG = dZ U / 2 and dU = 0) or
    32 (s = 1 in FP32, dU = 32 dZ, dG = dZ U), U and dZ even and small, X and W up to 1, all sums below 2^24."""
    g = 32.0 * rng.integers(0, 2, (M, N))
    u, dz = 2 * ints(rng, (M, N), 2), ints(rng, (M, N), 1)
    x, wg, wu = ints(rng, (M, K), 1), ints(rng, (K, N), 1), ints(rng, (K, N), 1)
    dg, du = np.where(g == 0, dz * u / 2, dz * u), np.where(g == 0, 0.0, 32 * dz)
    return x, wg, wu, g, u, dz, dg, du


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("dtype,pad,shift", [("bf16", 0, 0), ("f16", 8, 0), ("bf16", 3, 1), ("f16", 0, 4)])
def test_backward_stored(h, layout, M, N, K, dtype, pad, shift):
    say("gated_backward", layout, M, N, K, dtype, pad, shift)
    rng = np.random.default_rng(M + 3 * N + 5 * K)
    x, wg, wu, g, u, dz, dg, du = exact_case(rng, M, N, K)
    b = Block(h, layout, M, N, K, dtype, x, wg, wu, pad, shift)
    gd, ud, zd = (wide(v, N + pad, dtype, shift) for v in (g, u, dz))
    want = [dg @ wg.T + du @ wu.T, x.T @ dg, x.T @ du]
    outs = b.backward(zd, gd, ud)
    torch.cuda.synchronize()
    for a, w in zip(b.grads(outs), want):
        assert np.array_equal(a, rounded(w, dtype))
    # beta: the gradients accumulate onto 3 and -2 (halves of integers: exact before their one rounding).
    again = b.backward(zd, gd, ud, beta=0.5)
    torch.cuda.synchronize()
    for a, w in zip(b.grads(again), [want[0], want[1] + 1.5, want[2] - 1.0]):
        assert np.array_equal(a, rounded(w, dtype))
    # One half only: the other is not written.
    only = b.backward(zd, gd, ud, dw=False)
    torch.cuda.synchronize()
    assert torch.equal(only[0], outs[0]) and (only[1] == 3.0).all() and (only[2] == -2.0).all()
    only = b.backward(zd, gd, ud, dx=False)
    torch.cuda.synchronize()
    assert torch.equal(only[1], outs[1]) and torch.equal(only[2], outs[2]) and (only[0] == 7.0).all()


def backward_bounds(x, wg, wu, g, u, dz, dtype):
    """The oracle's gradients and how far the kernels' may be off: dG and dU computed in FP32 (sigmoid within 2e-6
    relative, six operations) and rounded once, then the products' sums and one rounding."""
    M, N = g.shape
    s = gated.sigmoid(g)
    dg, du = gated.pointwise(g, u, dz)
    # 1 - s is off by s's error; its share of dG is |dz u s g| of that.
    eg = (EPS[dtype] + 1e-5) * np.abs(dg) + 1e-5 * np.abs(dz * u * s) * (1 + np.abs(g)) + TINY[dtype]
    eu = (EPS[dtype] + 1e-5) * np.abs(du) + TINY[dtype]
    out = []
    for y, mag, err, terms in (
            (dg @ wg.T + du @ wu.T, np.abs(dg) @ np.abs(wg).T + np.abs(du) @ np.abs(wu).T,
             eg @ np.abs(wg).T + eu @ np.abs(wu).T, 2 * N),
            (x.T @ dg, np.abs(x).T @ np.abs(dg), np.abs(x).T @ eg, M),
            (x.T @ du, np.abs(x).T @ np.abs(du), np.abs(x).T @ eu, M)):
        out.append((y, err + EPS[dtype] * (np.abs(y) + err) + (terms + 2) * F32 * (mag + err) + TINY[dtype]))
    return out


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(20, 77, 130), (260, 333, 515), (700, 96, 200)])
def test_backward_random(h, layout, dtype, M, N, K):
    rng = np.random.default_rng(M)
    x, wg, wu, g, u, dz = (rounded(v, dtype) for v in (
        rng.standard_normal((M, K)), rng.standard_normal((K, N)) / np.sqrt(K), rng.standard_normal((K, N)) / np.sqrt(K),
        4 * rng.standard_normal((M, N)), rng.standard_normal((M, N)), rng.standard_normal((M, N))))
    b = Block(h, layout, M, N, K, dtype, x, wg, wu)
    got = b.grads(b.backward(*(wide(v, N, dtype) for v in (dz, g, u))))
    for a, (y, lim) in zip(got, backward_bounds(x, wg, wu, g, u, dz, dtype)):
        assert (np.abs(a - y) <= lim).all(), np.abs(a - y).max()


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (5, 40, 64), (31, 97, 40), (130, 260, 200), (257, 96, 515)])
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("dtype,pad", [("bf16", 0), ("f16", 3)])
def test_backward_again(h, layout, M, N, K, dtype, pad):
    """G and U computed again: from quarters of integers, so that the sums are exact and rounded as if stored."""
    say("gated_backward again", layout, M, N, K, dtype, pad)
    rng = np.random.default_rng(M + N + K)
    x, wg, wu = ints(rng, (M, K), 2) / 4, ints(rng, (K, N), 3) / 4, ints(rng, (K, N), 3) / 4
    dz = rounded(rng.standard_normal((M, N)), dtype)
    g, u = rounded(x @ wg, dtype), rounded(x @ wu, dtype)
    b = Block(h, layout, M, N, K, dtype, x, wg, wu, pad)
    zd = wide(dz, N + pad, dtype)
    limits = backward_bounds(x, wg, wu, g, u, dz, dtype)

    def check(outs, which=(0, 1, 2)):
        got = b.grads(outs)
        for i in which:
            y, lim = limits[i]
            assert (np.abs(got[i] - y) <= lim).all(), (i, np.abs(got[i] - y).max())
    check(b.backward(zd))
    # The same G and U stored by the forward pass (another order of sums, perhaps), and each half alone.
    _, gd, ud = b.forward()
    check(b.backward(zd, gd, ud))
    check(b.backward(zd, dw=False), (0,))
    check(b.backward(zd, dx=False), (1, 2))


@pytest.mark.parametrize("size", [128, 256])
@pytest.mark.parametrize("ksplit", [1, 2, 5, 32])
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("M,N,K", [(300, 424, 616), (130, 520, 1096)])
def test_every_tile(h, size, ksplit, layout, M, N, K):
    """Each product in each tile size and split, with tails of the contraction (sizes that are multiples of 8)."""
    say("gated tile", size, ksplit, layout, M, N, K)
    rng = np.random.default_rng(size + ksplit)
    x, wg, wu, g, u, dz, dg, du = exact_case(rng, M, N, K)
    want = [dg @ wg.T + du @ wu.T, x.T @ dg, x.T @ du]
    for dtype in ("bf16", "f16"):
        b = Block(h, layout, M, N, K, dtype, x, wg, wu)
        args = [wide(v, N, dtype) for v in (dz, g, u)]
        try:
            for p in range(3):
                mg.mgemm_set_gated_tile(h, p, size, ksplit)
            z, gd, ud = b.forward()
            outs = b.backward(*args)
            plus = b.backward(*args, beta=2.0)
            torch.cuda.synchronize()
        finally:
            for p in range(3):
                mg.mgemm_set_gated_tile(h, p)
        zo, go, uo = gated.forward(x, wg, wu)
        assert np.array_equal(gd.double().cpu().numpy(), rounded(go, dtype))
        assert np.array_equal(ud.double().cpu().numpy(), rounded(uo, dtype))
        zs = z.double().cpu().numpy()
        fits = np.abs(zo) < float(torch.finfo(TORCH[dtype]).max) * (1 - 2 * EPS[dtype])
        assert (np.abs(zs - zo)[fits] <= ((EPS[dtype] + 4e-6) * np.abs(zo) + TINY[dtype])[fits]).all()
        for a, w in zip(b.grads(outs), want):
            assert np.array_equal(a, rounded(w, dtype))
        for a, w in zip(b.grads(plus), [want[0], want[1] + 6.0, want[2] - 4.0]):
            assert np.array_equal(a, rounded(w, dtype))


# Sizes that take both tiles, whole and split contractions, with tails.
@pytest.mark.parametrize("M,N,K", [(1024, 1536, 1100), (2100, 5000, 520), (515, 2048, 4100), (4100, 300, 1030),
                                   (3000, 3100, 1000)])
@pytest.mark.parametrize("layout", ["row", "col"])
def test_larger(h, layout, M, N, K):
    say("gated larger", layout, M, N, K)
    gen = torch.Generator(device="cuda").manual_seed(M)

    def pick(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda").double()
    x, wg, wu = pick(-1, 1, M, K), pick(-1, 1, K, N), pick(-1, 1, K, N)
    b = Block(h, layout, M, N, K, "bf16", x, wg, wu)
    z, g, u = b.forward()
    go, uo = x @ wg, x @ wu
    assert torch.equal(g, go.bfloat16()) and torch.equal(u, uo.bfloat16())
    zo = go * torch.sigmoid(go) * uo
    assert ((z.double() - zo).abs() <= (EPS["bf16"] + 4e-6) * zo.abs() + TINY["bf16"]).all()
    g, u, dz = 32 * pick(0, 1, M, N), 2 * pick(-1, 1, M, N), pick(-1, 1, M, N)
    dg, du = torch.where(g == 0, dz * u / 2, dz * u), torch.where(g == 0, 0.0, 32 * dz)
    outs = b.backward(*(v.bfloat16() for v in (dz, g, u)))
    dwg, dwu = x.t() @ dg, x.t() @ du
    want = [dg @ wg.t() + du @ wu.t()] + ([dwg, dwu] if layout == "row" else [dwg.t(), dwu.t()])
    for a, w in zip(outs, want):
        assert torch.equal(a, w.bfloat16())


def test_far_gates(h):
    # |G| up to the type's largest: the gradients of a saturated or closed gate, no overflow in between.
    M, N, K = 8, 64, 8
    for dtype, far in (("f16", [-65504.0, -300.0, -30.0, 30.0, 300.0, 65504.0, -0.0, 0.0]),
                       ("bf16", [-3e38, -300.0, -30.0, 30.0, 300.0, 1e4, -0.0, 0.0])):
        g = rounded(np.repeat(np.array(far)[:, None], N, 1), dtype)
        u, dz = np.full((M, N), 0.5), np.zeros((M, N))
        for i in range(M):
            dz[i, i] = 1.0
        x, w = np.eye(M, K), np.zeros((K, N))
        b = Block(h, "row", M, N, K, dtype, x, w, w)
        _, dwg, dwu = b.grads(b.backward(*(wide(v, N, dtype) for v in (dz, g, u))))
        dg, du = gated.pointwise(g, u, dz)
        for got, ref in ((dwg, dg), (dwu, du)):
            assert np.isfinite(got).all()
            assert (np.abs(got - ref) <= (EPS[dtype] + 1e-4) * np.abs(ref) + 2 * TINY[dtype] + 1e-37).all()


def test_nan_reaches_its_row_and_columns_only(h):
    M, N, K = 70, 100, 90
    rng = np.random.default_rng(3)
    x, wg, wu, g, u, dz, dg, du = exact_case(rng, M, N, K)
    b = Block(h, "row", M, N, K, "bf16", x, wg, wu)
    dz[11, 42] = np.nan
    dx, dwg, dwu = b.grads(b.backward(*(wide(v, N, "bf16") for v in (dz, g, u))))
    assert np.isnan(dx[11]).all() and not np.isnan(np.delete(dx, 11, 0)).any()
    for d in (dwg, dwu):
        assert np.isnan(d[:, 42]).all() and not np.isnan(np.delete(d, 42, 1)).any()


def test_empty_sizes(h):
    for layout in ("row", "col"):
        for M, N, K in ((0, 16, 24), (16, 0, 24)):
            b = Block(h, layout, M, N, K, "bf16", np.zeros((M, K)), np.zeros((K, N)), np.zeros((K, N)), pad=8)
            b.forward()
            e = torch.zeros(max(M, 1), max(N, 1), dtype=torch.bfloat16, device="cuda")
            outs = b.backward(e, e, e, beta=2.0)
            torch.cuda.synchronize()
            dx, dwg, dwu = b.grads(outs)
            assert (dx == 0).all() and (dwg == 6.0).all() and (dwu == -4.0).all()
        b = Block(h, layout, 5, 16, 0, "f16", np.zeros((5, 0)), np.zeros((0, 16)), np.zeros((0, 16)), pad=8)
        z, g, u = b.forward()
        torch.cuda.synchronize()
        for t in (z, g, u):
            assert (t[:, :16] == 0).all() and (t[:, 16:] == 7.0).all()


def test_other_stream_and_graph(h):
    # Calls on a stream that is not the current one, and replays of captured passes, against the eager results.
    M, N, K = 300, 416, 1000
    rng = np.random.default_rng(5)
    x, wg, wu, g, u, dz = (rng.standard_normal(s) / d for s, d in (((M, K), 1), ((K, N), 30), ((K, N), 30), ((M, N), 1),
                                                                 ((M, N), 1), ((M, N), 1)))
    b = Block(h, "row", M, N, K, "bf16", x, wg, wu)
    zd, gd, ud = (wide(v, N, "bf16") for v in (dz, g, u))
    side = torch.cuda.Stream()
    for stored in (True, False):
        args = (zd, gd, ud) if stored else (zd,)
        want_f, want_b = b.forward(), b.backward(*args)
        torch.cuda.synchronize()
        fo, bo = b.forward(stream=side), None
        keep = b.kept
        bo = b.backward(*args, stream=side)
        side.synchronize()
        for a, c in zip(fo + tuple(bo), want_f + tuple(want_b)):
            assert torch.equal(a, c)
        del keep
        work = b.work(True, stored)
        outs = [t.clone() for t in want_b]
        fouts = [t.clone() for t in want_f]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.forward(outs=fouts)
            fkeep = b.kept
            b.backward(*args, outs=outs)
            bkeep = b.kept
        for i in range(3):
            b.x.mul_(-0.5)
            zd.mul_(2.0)
            want_f, want_b = b.forward(), b.backward(*args)
            torch.cuda.synchronize()
            for t in outs + fouts:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for a, c in zip(fouts + outs, list(want_f) + list(want_b)):
                assert torch.equal(a, c), i
        del work, fkeep, bkeep


def test_offsets_past_31_bits(h):
    # 66000 x 33000 outputs: element and byte offsets beyond 2^31, in and out.
    M, N, K = 66000, 33000, 64
    gen = torch.Generator(device="cuda").manual_seed(2)

    def pick(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    say("gated large", M, N, K)
    x, wg, wu = pick(-1, 1, M, K), pick(-1, 1, K, N), pick(-1, 1, K, N)
    z, g, u = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    w = torch.empty(mg.mgemm_gated_workspace("row", M, N, K, x, K, wg, wu, N, "bf16", True, True), dtype=torch.uint8,
                    device="cuda")
    mg.mgemm_gated_forward(h, "row", M, N, K, x, K, wg, wu, N, z, N, g, u, N, "bf16", w, w.numel())
    dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)
    # Sums of up to 64 units are exact in BF16; the backward pass takes G = 0 or 32 (see exact_case).
    for m in range(0, M, 6000):
        go, uo = x[m:m + 6000].float() @ wg.float(), x[m:m + 6000].float() @ wu.float()
        assert torch.equal(g[m:m + 6000].float(), go) and torch.equal(u[m:m + 6000].float(), uo)
        zo = go.double() * torch.sigmoid(go.double()) * uo.double()
        assert ((z[m:m + 6000].double() - zo).abs() <= (EPS["bf16"] + 4e-6) * zo.abs() + TINY["bf16"]).all()
        del go, uo, zo
    dz = z
    for m in range(0, M, 6000):
        g[m:m + 6000] = 32 * pick(0, 1, min(6000, M - m), N)
        dz[m:m + 6000] = pick(-1, 1, min(6000, M - m), N)
        u[m:m + 6000] = 2 * pick(-1, 1, min(6000, M - m), N)
    mg.mgemm_gated_backward(h, "row", M, N, K, x, K, wg, wu, N, g, u, N, dz, N, dx, K, dwg, dwu, N, 0.0, "bf16", w,
                            w.numel())
    og, ou = torch.zeros(K, N, device="cuda", dtype=torch.float64), torch.zeros(K, N, device="cuda", dtype=torch.float64)
    for m in range(0, M, 6000):
        gs, us, ds, xs = (t[m:m + 6000].float() for t in (g, u, dz, x))
        dg, du = torch.where(gs == 0, ds * us / 2, ds * us), torch.where(gs == 0, 0.0, 32 * ds)
        # Products of integers, sums below 2^24: exact in 32 bits.
        assert torch.equal(dx[m:m + 6000], (dg @ wg.float().t() + du @ wu.float().t()).bfloat16())
        og += (xs.t() @ dg).double()
        ou += (xs.t() @ du).double()
        del gs, us, ds, dg, du
    assert torch.equal(dwg, og.bfloat16()) and torch.equal(dwu, ou.bfloat16())


def test_example_trains_and_serves():
    import examples.gated_block as example
    losses, off = example.main(steps=30)
    assert losses[-1] < 0.6 * losses[0]
    # E2M1 keeps about 3 bits of each operand: 10 to 20% of the norm for products of normal values.
    assert 0.01 < off < 0.35
