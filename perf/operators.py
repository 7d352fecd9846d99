"""The gated feed-forward block's operators, as they are measured: the 16-bit
block's forward and backward passes (training), and microscaled 4-bit
quantisation, product and gated pair (serving).

    quantize        X (M x K) to E2M1 codes in blocks of 32 with E8M0 scales, read back
    linear          Y = Q(X) W^T with 4-bit weights and activations quantised in the call
    gated           Z = SiLU(Q(X) Wg^T) * (Q(X) Wu^T) with 4-bit weights
    gated_forward   G = X Wg, U = X Wu, Z = SiLU(G) * U, all three stored
    gated_backward  dX, dWg, dWu from dZ, with G and U stored or computed again

`own` False: plain torch operations in 32 bits; True: the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 32
# Products of the largest drawn case, by kind: those of the largest listed one.
MOST = {"quantize": 12288 * 4096, "linear": 8192 * 12288 * 4096, "gated": 2 * 1024 * 12288 * 4096,
        "gated_forward": 2 * 1024 * 12288 * 4096, "gated_backward": 4 * 1024 * 12288 * 4096}
FACTOR = {"quantize": 1, "linear": 1, "gated": 2, "gated_forward": 2, "gated_backward": 4}


def listed():
    return [
        # A step's activations of a small decode batch.
        dict(name="quantize_batch16", kind="quantize", M=16, K=4096, dtype="bf16", pad=0),
        # An FP32 master weight made into the 4-bit weight that is served (12288 x 4096).
        dict(name="quantize_weight_f32", kind="quantize", M=12288, K=4096, dtype="f32", pad=0),
        # One token through the up projection: latency, bound by the weights' bytes.
        dict(name="linear_decode_1", kind="linear", M=1, N=12288, K=4096, dtype="bf16", pad=0),
        # A batch of tokens through the down projection.
        dict(name="linear_batch_48", kind="linear", M=48, N=4096, K=12288, dtype="f16", pad=0),
        # A long prompt (or many of them) through the up projection.
        dict(name="linear_prompt_8192", kind="linear", M=8192, N=12288, K=4096, dtype="bf16", pad=0),
        # A few tokens through the gated pair.
        dict(name="gated_decode_4", kind="gated", M=4, N=12288, K=4096, dtype="bf16", pad=0),
        # A prompt through the gated pair.
        dict(name="gated_prompt_1024", kind="gated", M=1024, N=12288, K=4096, dtype="bf16", pad=0),
        # Training: one GPU's eighth of the block's columns.
        dict(name="forward_share_1536", kind="gated_forward", M=1024, N=1536, K=4096, dtype="bf16", pad=0, layout="row"),
        # Training: ragged sizes, weights stored out x in, rows of a wider tensor.
        dict(name="forward_ragged_col", kind="gated_forward", M=777, N=1000, K=1001, dtype="f16", pad=3, layout="col"),
        # Training: the whole block's backward pass from the stored G and U.
        dict(name="backward_ffn", kind="gated_backward", M=1024, N=12288, K=4096, dtype="bf16", pad=0, layout="row", stored=True),
        # Training: ragged sizes, G and U computed again to save memory.
        dict(name="backward_ragged_again", kind="gated_backward", M=333, N=1004, K=515, dtype="f16", pad=0, layout="row", stored=False),
        # Training: weights stored out x in, an eighth of the columns.
        dict(name="backward_share_col", kind="gated_backward", M=1024, N=1536, K=4096, dtype="bf16", pad=0, layout="col", stored=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(sorted(MOST))
    serving = kind in ("quantize", "linear", "gated")
    K, N, M = _log(rng, 33, 12288), _log(rng, 17, 12288), _log(rng, 1 if serving else 16, 8192)
    if rng.random() < 0.5:  # the sizes that models have: multiples of 64
        K, N = max(64, K // 64 * 64), max(64, N // 64 * 64)
    case = dict(kind=kind, M=M, K=K, dtype=rng.choice(["bf16", "f16", "f32"] if kind == "quantize" else ["bf16", "f16"]),
                pad=rng.choice([0, 0, 8, 3]))
    if kind != "quantize":
        case["N"] = N
    if kind.startswith("gated_"):
        case["layout"] = rng.choice(["row", "col"])
    if kind == "gated_backward":
        case["stored"] = rng.random() < 0.7
    cost = FACTOR[kind] * M * K * case.get("N", 1)
    if cost > MOST[kind]:
        case["M"] = max(1, M * MOST[kind] // cost)
    return case


def _pitch(K):
    """Bytes of a row of scales: a byte for each block of 32, rounded up to 16."""
    return -(-K // (16 * BLOCK)) * 16


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    M, K, N, dt = case["M"], case["K"], case.get("N", 0), DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    # Activations: normal, with a few channels eight times the others; a view of a wider tensor where pad > 0.
    x = normal(M, K + case["pad"])
    x *= 1.0 + 7.0 * (torch.rand(K + case["pad"], generator=gen, device="cuda") < 0.01)
    s = {"case": case, "x": x.to(dt)[:, :K]}
    if case["kind"] == "quantize":
        s["codes"] = torch.empty(M, -(-K // BLOCK) * 16, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(M, _pitch(K), dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty(M, K, dtype=dt, device="cuda")
    elif case["kind"] in ("linear", "gated"):
        names = ["w"] if case["kind"] == "linear" else ["wg", "wu"]
        for name in names:
            codes, scales = _codes(_blocks(normal(N, K) / math.sqrt(K)))
            s[name] = (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()
            s[name + "_scales"] = torch.zeros(N, _pitch(K), dtype=torch.uint8, device="cuda")
            s[name + "_scales"][:, :scales.shape[1]] = scales
        s["y"] = torch.empty(M, N, dtype=dt, device="cuda")
    else:
        # Weights in x out, stored by rows or (out x in) by columns: s["wg"] is always the stored tensor.
        shape = (K, N) if case["layout"] == "row" else (N, K)
        s["wg"], s["wu"] = ((normal(*shape) / math.sqrt(K)).to(dt) for _ in range(2))
        if case["kind"] == "gated_forward":
            s["out"] = [torch.empty(M, N, dtype=dt, device="cuda") for _ in range(3)]
        else:
            s["dz"] = (0.5 * normal(M, N)).to(dt)
            if case["stored"]:
                wg, wu = (w.float() if case["layout"] == "row" else w.float().t() for w in (s["wg"], s["wu"]))
                s["g"], s["u"] = (s["x"].float() @ wg).to(dt), (s["x"].float() @ wu).to(dt)
            s["out"] = [torch.empty(M, K, dtype=dt, device="cuda"), torch.empty_like(s["wg"]), torch.empty_like(s["wu"])]
    return s


# --- the plain form -------------------------------------------------------

def _blocks(x):
    """x (rows x K) in 32 bits, zeros up to a whole block of 32."""
    x = x.float()
    return torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK))


def _codes(x):
    """E2M1 codes (one to a byte) and E8M0 scale bytes of x (rows x a multiple of 32)."""
    b = x.view(x.shape[0], -1, BLOCK)
    top = b.abs().amax(2)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 127)
    t = torch.ldexp(b, -e[:, :, None])
    a = t.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    v = (torch.round(a / step) * step).clamp(max=6.0)
    code = torch.where(v < 2, 2 * v, torch.where(v < 4, v + 2, v / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(t).to(torch.uint8) << 3)
    return code.reshape(x.shape), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """The values that codes (one to a byte) and scale bytes stand for."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    v = table[(codes & 7).int()] * (1.0 - 2.0 * (codes >> 3).float())
    v = torch.ldexp(v.view(codes.shape[0], -1, BLOCK), scales[:, :, None].int() - 127)
    return v.view(codes.shape)


def _weight(s, name):
    packed = s[name]
    codes = torch.stack([packed & 15, packed >> 4], 2).view(packed.shape[0], -1)
    return _values(codes, s[name + "_scales"][:, :codes.shape[1] // BLOCK])


def _plain(s):
    case, x = s["case"], s["x"]
    kind, dt, K = case["kind"], x.dtype, case["K"]
    if kind == "quantize":
        return _values(*_codes(_blocks(x)))[:, :K].to(dt)
    if kind in ("linear", "gated"):
        q = _values(*_codes(_blocks(x)))
        if kind == "linear":
            return (q @ _weight(s, "w").t()).to(dt)
        g, u = q @ _weight(s, "wg").t(), q @ _weight(s, "wu").t()
        return (g / (1 + torch.exp(-g)) * u).to(dt)
    xf, row = x.float(), case["layout"] == "row"
    wg, wu = (w.float() if row else w.float().t() for w in (s["wg"], s["wu"]))
    if kind == "gated_forward":
        g, u = xf @ wg, xf @ wu
        return [(g / (1 + torch.exp(-g)) * u).to(dt), g.to(dt), u.to(dt)]
    # Without stored G and U they are what the forward pass would have stored.
    g, u = (s["g"].float(), s["u"].float()) if case["stored"] else ((xf @ wg).to(dt).float(), (xf @ wu).to(dt).float())
    dz = s["dz"].float()
    sig = 1 / (1 + torch.exp(-g))
    du, dg = dz * g * sig, dz * u * sig * (1 + g * (1 - sig))
    dx = dg @ wg.t() + du @ wu.t()
    dwg, dwu = (xf.t() @ dg, xf.t() @ du) if row else (dg.t() @ xf, du.t() @ xf)
    return [dx.to(dt), dwg.to(dt), dwu.to(dt)]


# --- the library ----------------------------------------------------------

_library = []


def _handle():
    if not _library:
        import dense_gemm_mgemm_amd as mg
        _library.extend([mg, mg.mgemm_create(), {}])
    return _library


def _own(s):
    mg, h, workspaces = _handle()
    case, x = s["case"], s["x"]
    kind, M, K, N, dt, ldx = case["kind"], case["M"], case["K"], case.get("N", 0), case["dtype"], x.stride(0)
    if kind == "quantize":
        q, sc, y = s["codes"], s["scales"], s["y"]
        mg.mgemm_quantize_mx4(h, M, K, x, ldx, dt, q, q.stride(0), sc, sc.stride(0))
        mg.mgemm_dequantize_mx4(h, M, K, q, q.stride(0), sc, sc.stride(0), y, K, dt)
        return y
    if kind == "linear":
        mg.mgemm_linear_mx4(h, M, N, K, x, ldx, dt, s["w"], s["w"].stride(0), s["w_scales"], s["w_scales"].stride(0),
                            s["y"], N, dt)
        return s["y"]
    if kind == "gated":
        mg.mgemm_gated_mx4(h, M, N, K, x, ldx, dt, s["wg"], s["wg_scales"], s["wu"], s["wu_scales"], s["wg"].stride(0),
                           s["wg_scales"].stride(0), s["y"], N, dt)
        return s["y"]
    layout, ldw = case["layout"], s["wg"].stride(0)
    # One workspace for each size, kept and used again as a training loop does.
    backward, stored = kind == "gated_backward", case.get("stored", False)
    key = (kind, layout, stored, M, N, K, ldx, dt)
    if key not in workspaces:
        size = mg.mgemm_gated_workspace(layout, M, N, K, x, ldx, s["wg"], s["wu"], ldw, dt, backward, stored)
        workspaces.clear()
        workspaces[key] = torch.empty(size, dtype=torch.uint8, device="cuda")
    w = workspaces[key]
    if not backward:
        z, g, u = s["out"]
        mg.mgemm_gated_forward(h, layout, M, N, K, x, ldx, s["wg"], s["wu"], ldw, z, N, g, u, N, dt, w, w.numel())
        return [z, g, u]
    dx, dwg, dwu = s["out"]
    mg.mgemm_gated_backward(h, layout, M, N, K, x, ldx, s["wg"], s["wu"], ldw, s.get("g"), s.get("u"), N, s["dz"], N,
                            dx, K, dwg, dwu, ldw, 0.0, dt, w, w.numel())
    return [dx, dwg, dwu]


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    kind, M, K, N, b = case["kind"], case["M"], case["K"], case.get("N", 0), BYTES[case["dtype"]]
    mx4 = -(-K // BLOCK) * 17  # bytes of K codes and their scales
    if kind == "quantize":
        # Read X, write the codes and scales, and the values read back.
        return {"bytes": 2 * M * K * b + M * mx4, "flops": 2 * M * K}
    if kind == "linear":
        return {"bytes": M * K * b + N * mx4 + M * N * b, "flops": 2 * M * N * K}
    if kind == "gated":
        return {"bytes": M * K * b + 2 * N * mx4 + M * N * b, "flops": 4 * M * N * K}
    if kind == "gated_forward":
        return {"bytes": (M * K + 2 * K * N + 3 * M * N) * b, "flops": 4 * M * N * K}
    again = 0 if case["stored"] else 4
    return {"bytes": (2 * M * K + 4 * K * N + M * N + (2 * M * N if case["stored"] else 0)) * b, "flops": (8 + again) * M * N * K}


# --- the definition in 64 bits --------------------------------------------

def _nearest(x):
    """x (rows x K, 64 bits) rounded to the microscaled 4-bit values of its blocks."""
    rows, K = x.shape
    full = torch.zeros(rows, -(-K // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    full[:, :K] = x
    b = full.reshape(-1, BLOCK)
    top = b.abs().max(1, keepdim=True).values
    scale = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -125))) - 2)
    a = b.abs() / scale
    grid = a.new_tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    # The border between neighbours i and i + 1 belongs to the even one.
    up = torch.zeros_like(a, dtype=torch.int64)
    for i in range(7):
        border = (grid[i] + grid[i + 1]) / 2
        up += (a > border) if i % 2 == 0 else (a >= border)
    return (torch.sign(b) * grid[up] * scale).reshape(rows, -1)[:, :K]


def _stored_values(s, name, K):
    low = s[name].to(torch.int64)
    nibbles = torch.empty(low.shape[0], 2 * low.shape[1], dtype=torch.int64, device=low.device)
    nibbles[:, 0::2], nibbles[:, 1::2] = low % 16, low // 16
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=low.device)
    power = torch.exp2(s[name + "_scales"][:, :nibbles.shape[1] // BLOCK].double() - 127)
    return (grid[nibbles] * power.repeat_interleave(BLOCK, dim=1))[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    kind, K = case["kind"], case["K"]
    x = s["x"].double()
    if kind == "quantize":
        return _nearest(x)
    if kind == "linear":
        return torch.mm(_nearest(x), _stored_values(s, "w", K).T)
    if kind == "gated":
        q = _nearest(x)
        g = torch.mm(q, _stored_values(s, "wg", K).T)
        return g * torch.sigmoid(g) * torch.mm(q, _stored_values(s, "wu", K).T)
    wg, wu = (s[n].double() if case["layout"] == "row" else s[n].double().T for n in ("wg", "wu"))
    if kind == "gated_forward":
        g, u = torch.mm(x, wg), torch.mm(x, wu)
        return [g * torch.sigmoid(g) * u, g, u]
    if case["stored"]:
        g, u = s["g"].double(), s["u"].double()
    else:
        g, u = (torch.mm(x, w).to(s["x"].dtype).double() for w in (wg, wu))
    sig, dz = torch.sigmoid(g), s["dz"].double()
    dsilu = sig + g * sig * (1 - sig)
    dg, du = dz * u * dsilu, dz * g * sig
    dx = torch.mm(dg, wg.T) + torch.mm(du, wu.T)
    dwg, dwu = torch.mm(x.T, dg), torch.mm(x.T, du)
    return [dx, dwg, dwu] if case["layout"] == "row" else [dx, dwg.T, dwu.T]
