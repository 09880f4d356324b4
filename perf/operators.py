"""Measured cases of the operators around an NVFP4 linear layer.

Four operators, each in its plain form (elementary torch operations in fp32)
and as the calls that a program makes of this package:

  sandwich  post-norm of a block's output, gate and residual scale, residual
            add, pre-norm of the next block, quantization (or y alone)
  quantize  a 16-bit matrix to NVFP4 (codes and swizzled block scales) and
            back to 16 bits, the round trip of weight preparation and of
            simulated quantization
  gated     the activation between the two products of a gated MLP,
            act(gate) * up, quantized for the down projection
  linear    the product of an NVFP4 activation with an NVFP4 weight

Packed 4-bit codes are returned as the values they stand for: they go
through the package's dequantization, into E4M3 where the quantized values
are computed rather than given (a last-place difference of the activation
may move a code by a step there).
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
# E2M1 magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6: the borders between neighbours
# (a tie goes to the even code) and the step across each.
E2M1_BORDERS = ((0.25, False, 0.5), (0.75, True, 0.5), (1.25, False, 0.5), (1.75, True, 0.5),
                (2.5, False, 1.0), (3.5, True, 1.0), (5.0, False, 2.0))
E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one token of a decode step: latency
        dict(name="sandwich_m1_h2048_fp8", op="sandwich", M=1, H=2048, dtype="bf16", mode="fp8",
             gate="none", res_scale=1.0),
        # a decode batch with one gate per token, the normed y kept in 16 bits
        dict(name="sandwich_m256_h4096_y_gated", op="sandwich", M=256, H=4096, dtype="bf16",
             mode="none", gate="rows", res_scale=1.0),
        # a prefill chunk into NVFP4, one gate per channel, a residual scale
        dict(name="sandwich_m2048_h5120_nvfp4", op="sandwich", M=2048, H=5120, dtype="bf16",
             mode="nvfp4", gate="channels", res_scale=0.22),
        # the largest prefill batch
        dict(name="sandwich_m16384_h8192_fp8", op="sandwich", M=16384, H=8192, dtype="fp16",
             mode="fp8", gate="none", res_scale=1.0),
        # a ragged handful of rows of a fused projection's output (a strided slice)
        dict(name="quantize_m33_k2048", op="quantize", M=33, K=2048, dtype="bf16", stride=2 * 2048),
        # a whole weight or a prefill batch
        dict(name="quantize_m16384_k8192", op="quantize", M=16384, K=8192, dtype="fp16", stride=8192),
        # the MLP's activation in a decode batch
        dict(name="gated_m16_h5120_gelu_fp8", op="gated", M=16, H=5120, dtype="bf16",
             mode="fp8", act="gelu_tanh"),
        # and in a prefill batch, for an NVFP4 down projection
        dict(name="gated_m4096_h7168_silu_nvfp4", op="gated", M=4096, H=7168, dtype="bf16",
             mode="nvfp4", act="silu"),
        # one token: the weight is read once, nothing else matters
        dict(name="linear_m1_n4096_k2048", op="linear", M=1, N=4096, K=2048, dtype="bf16", bias=False),
        # a decode batch
        dict(name="linear_m16_n8192_k5120", op="linear", M=16, N=8192, K=5120, dtype="bf16", bias=False),
        # a ragged middle size with a bias, rows and columns inside a tile
        dict(name="linear_m300_n5000_k4096", op="linear", M=300, N=5000, K=4096, dtype="fp16", bias=True),
        # a prefill batch
        dict(name="linear_m8192_n8192_k5120", op="linear", M=8192, N=8192, K=5120, dtype="bf16", bias=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("sandwich", "quantize", "gated", "linear", "linear"))
    dtype = rng.choice(("bf16", "fp16"))
    M = _log(rng, 1, 16384)
    if op == "sandwich":
        mode = rng.choice(("fp8", "nvfp4", "none"))
        H = 64 * _log(rng, 8, 128) if mode == "nvfp4" else 8 * _log(rng, 64, 1024)
        return dict(op=op, M=M, H=H, dtype=dtype, mode=mode,
                    gate=rng.choice(("none", "channels", "rows")), res_scale=rng.choice((1.0, 0.22, 1.5)))
    if op == "quantize":
        K = 64 * _log(rng, 8, 128)
        return dict(op=op, M=M, K=K, dtype=dtype, stride=K + rng.choice((0, 8, 64, K)))
    if op == "gated":
        mode = rng.choice(("fp8", "nvfp4", "none"))
        H = 64 * _log(rng, 8, 112) if mode == "nvfp4" else 8 * _log(rng, 64, 896)
        return dict(op=op, M=M, H=H, dtype=dtype, mode=mode, act=rng.choice(("silu", "gelu_tanh")))
    K = 64 * _log(rng, 4, 112)
    N = _log(rng, 64, 8192)
    M = min(M, 8192 * 8192 * 5120 // (N * K))
    return dict(op=op, M=M, N=N, K=K, dtype=dtype, bias=rng.random() < 0.5)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = DT[case["dtype"]]

    def normal(*shape, sd=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * sd

    def one(v):
        return torch.full((1,), v, dtype=torch.float32, device="cuda")

    s = dict(case)
    op, M = case["op"], case["M"]
    if op == "sandwich":
        H = case["H"]
        s["x"] = normal(M, H).to(T)
        r = normal(M, H, sd=3.0)
        r[:, torch.randperm(H, generator=g, device="cuda")[:8]] *= 20.0  # the residual stream's outlier channels
        s["residual"] = r.to(T)
        s["post"] = normal(H, sd=math.sqrt(0.1)).to(T)
        s["pre"] = normal(H, sd=math.sqrt(0.1)).to(T)
        s["gate_t"] = {"none": lambda: None, "channels": lambda: normal(H).to(T),
                       "rows": lambda: torch.tanh(normal(M, H)).to(T)}[case["gate"]]()
        s["scale"] = one({"fp8": 0.05, "nvfp4": 168.0, "none": 1.0}[case["mode"]])
        s["res_out"] = torch.empty_like(s["residual"])
        _outputs(s, M, H, case["mode"], T)
    elif op == "quantize":
        K = case["K"]
        s["x"] = normal(M, case["stride"], sd=1.5).to(T)[:, :K]
        s["scale"] = one(200.0)
        _outputs(s, M, K, "nvfp4", T)
        s["back"] = torch.empty(M, K, dtype=T, device="cuda")
    elif op == "gated":
        H = case["H"]
        s["x"] = normal(M, 2 * H).to(T)
        s["scale"] = one({"fp8": 0.02, "nvfp4": 250.0, "none": 1.0}[case["mode"]])
        _outputs(s, M, H, case["mode"], T)
    else:
        N, K = case["N"], case["K"]
        s["aq"], s["asf"] = _pack(*_nvfp4(normal(M, K).to(T), one(400.0)))
        s["bq"], s["bsf"] = _pack(*_nvfp4(normal(N, K, sd=0.03).to(T), one(16000.0)))
        s["alpha"] = one(1.0 / (400.0 * 16000.0))
        s["bias_t"] = normal(N).to(T) if case["bias"] else None
        s["y"] = torch.empty(M, N, dtype=T, device="cuda")
    return s


def _outputs(s, M, H, mode, T):
    """The output buffers that a program keeps: scale padding rows are never written."""
    s["y"] = torch.empty(M, H, dtype=T, device="cuda") if mode == "none" else None
    s["q"] = s["sf"] = None
    if mode == "fp8":
        s["q"] = torch.empty(M, H, dtype=E4M3, device="cuda")
    if mode == "nvfp4":
        s["q"] = torch.empty(M, H // 2, dtype=torch.uint8, device="cuda")
        s["sf"] = torch.zeros(-(-M // 128) * 128, H // 16, dtype=torch.uint8, device="cuda").view(E4M3)
        s["e4m3"] = torch.empty(M, H, dtype=E4M3, device="cuda")


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _e2m1(v):
    """The E2M1 value nearest to v (ties to the even code, saturating at 6)."""
    a = v.abs()
    r = torch.zeros_like(a)
    for border, tie_up, step in E2M1_BORDERS:
        r = r + step * ((a >= border) if tie_up else (a > border)).to(a.dtype)
    return torch.copysign(r, v)


def _e4m3(v):
    return v.clamp(-448.0, 448.0).to(E4M3)


def _nvfp4(x, scale, wide=torch.float32):
    """(E2M1 values (M, K), E4M3 block scales (M, K/16)) of a 16-bit matrix."""
    M, K = x.shape
    b = x.to(wide).reshape(M, K // 16, 16)
    g = scale.to(wide)
    sf = _e4m3(g * (b.abs().amax(-1) / 6.0))
    v = sf.to(wide)
    es = torch.where(v > 0, g / torch.where(v > 0, v, torch.ones_like(v)), torch.zeros_like(v))
    return _e2m1(b * es[..., None]).reshape(M, K), sf


def _swizzle(sf):
    """(M, Kb) block scales in the 128x4 layout: (round_up(M, 128), Kb), padding 0."""
    M, Kb = sf.shape
    Mp = -(-M // 128) * 128
    p = torch.zeros(Mp, Kb, dtype=torch.uint8, device=sf.device)
    p[:M] = sf.view(torch.uint8)
    return p.reshape(Mp // 128, 4, 32, Kb // 4, 4).permute(0, 3, 2, 1, 4).reshape(Mp, Kb).view(E4M3)


def _unswizzle(sw, M):
    Mp, Kb = sw.shape
    p = sw.view(torch.uint8).reshape(Mp // 128, Kb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(Mp, Kb)
    return p[:M].view(E4M3)


def _pack(values, sf):
    a = values.abs()
    mag = torch.where(a <= 2.0, a * 2.0, torch.where(a == 6.0, a + 1.0, a + 2.0)).to(torch.uint8)
    code = mag | (torch.signbit(values).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), _swizzle(sf)


def _unpack(q, sw, wide=torch.float32):
    """code * block scale of packed NVFP4, exact in fp32."""
    M, half = q.shape
    lut = torch.tensor(E2M1_VALUES, dtype=wide, device=q.device)
    v = lut[torch.stack((q & 15, q >> 4), -1).to(torch.int32)].reshape(M, half // 8, 16)
    return (v * _unswizzle(sw, M).to(wide)[..., None]).reshape(M, 2 * half)


def _back(values, sf, scale, dtype):
    """code * (block scale / global scale), rounded to `dtype`."""
    M, K = values.shape
    v = values.reshape(M, K // 16, 16) * (sf.to(values.dtype) / scale.to(values.dtype))[..., None]
    v = v.reshape(M, K)
    return _e4m3(v) if dtype is E4M3 else v.to(dtype)


def _norm(v, w):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * (1.0 + w)


def _act(g, kind):
    if kind == "silu":
        return g / (1.0 + torch.exp(-g))
    return g / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _quantized(s, y, wide):
    """The outputs of one mode, from the rounded y."""
    if s["mode"] == "none":
        return (y,)
    if s["mode"] == "fp8":
        return (_e4m3(y.to(wide) / s["scale"].to(wide)),)
    values, sf = _nvfp4(y, s["scale"], wide)
    return _back(values, sf, s["scale"], E4M3), _swizzle(sf)


def _plain(s, wide=torch.float32):
    op, T = s["op"], DT[s["dtype"]]
    if op == "sandwich":
        u = _norm(s["x"].to(wide), s["post"].to(wide))
        if s["gate_t"] is not None:
            u = u * s["gate_t"].to(wide)
        h = (s["residual"].to(wide) + s["res_scale"] * u).to(T)
        y = _norm(h.to(wide), s["pre"].to(wide)).to(T)
        return (h, *_quantized(s, y, wide))
    if op == "quantize":
        values, sf = _nvfp4(s["x"], s["scale"], wide)
        return _back(values, sf, s["scale"], T), _swizzle(sf)
    if op == "gated":
        x = s["x"].to(wide)
        y = (_act(x[:, :s["H"]], s["act"]) * x[:, s["H"]:]).to(T)
        return _quantized(s, y, wide)
    y = _unpack(s["aq"], s["asf"], wide) @ _unpack(s["bq"], s["bsf"], wide).t() * s["alpha"].to(wide)
    if s["bias_t"] is not None:
        y = y + s["bias_t"].to(wide)
    return (y.to(T),)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    if own:
        import nvfp4_quant_gemma_gb300 as gnq
        op = s["op"]
        if op == "linear":
            return gnq.nvfp4_linear(s["aq"], s["asf"], s["bq"], s["bsf"], s["alpha"],
                                    bias=s["bias_t"], out=s["y"]),
        if op == "quantize":
            q, sf = gnq.quantize(s["x"], s["scale"], "nvfp4", out=(s["q"], s["sf"]))
            return gnq.nvfp4_dequantize(q, sf, s["scale"], out=s["back"]), sf
        if op == "sandwich":
            q, sf, y = gnq.gemma_sandwich_norm_quant(
                s["x"], s["residual"], s["post"], s["pre"], EPS, s["scale"], s["mode"], gate=s["gate_t"],
                residual_scale=s["res_scale"], residual_out=s["res_out"], out=(s["q"], s["sf"], s["y"]))
            first = (s["res_out"],)
        else:
            q, sf, y = gnq.gated_act_quant(s["x"], s["scale"], s["mode"], act=s["act"],
                                           out=(s["q"], s["sf"], s["y"]))
            first = ()
        if s["mode"] == "none":
            return (*first, y)
        if s["mode"] == "fp8":
            return (*first, q)
        return (*first, gnq.nvfp4_dequantize(q, sf, s["scale"], out=s["e4m3"]), sf)
    return _plain(s)


def work(case):
    op, M = case["op"], case["M"]
    if op == "linear":
        N, K = case["N"], case["K"]
        return dict(bytes=(M + N) * K * 9 / 16 + 2 * M * N + (2 * N if case["bias"] else 0), flops=2 * M * N * K)
    n = M * (case["K"] if op == "quantize" else case["H"])
    nvfp4 = n * 9 / 16  # codes and block scales: written by one call, read by the next
    if op == "quantize":
        return dict(bytes=2 * n + 2 * nvfp4 + 2 * n, flops=8 * n)
    out = {"none": 2 * n, "fp8": n, "nvfp4": 2 * nvfp4 + n}[case["mode"]]
    if op == "gated":
        return dict(bytes=4 * n + out, flops=12 * n)
    gate = {"none": 0, "channels": 2 * case["H"], "rows": 2 * n}[case["gate"]]
    return dict(bytes=6 * n + 4 * case["H"] + gate + out, flops=14 * n)


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    """Outputs from the definitions in fp64.  The 4-bit and 8-bit steps pick the
    nearest of all code values by search, and scales are placed by the layout's
    byte formula, unlike the plain forms."""
    s = prepare(case, seed)
    f64, T, M = torch.float64, DT[case["dtype"]], case["M"]
    e2 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=f64, device="cuda")
    e4 = torch.arange(127, dtype=torch.uint8, device="cuda").view(E4M3).to(f64)  # 0 .. 448, ascending

    def nearest(v, values):
        """Index of the value nearest to |v|: the lower neighbour, or the upper one where it is nearer or a tie's even code."""
        a = v.abs().clamp(max=float(values[-1]))
        lo = (torch.searchsorted(values, a, right=True) - 1).clamp(0, len(values) - 2)
        down, up = a - values[lo], values[lo + 1] - a
        return lo + ((up < down) | ((up == down) & (lo % 2 == 1))).to(lo.dtype)

    def to_e4m3(v):
        c = nearest(v, e4).to(torch.uint8)
        return (c | (torch.signbit(v).to(torch.uint8) << 7)).view(E4M3)

    def offsets(rows, Kb):
        m = torch.arange(rows, device="cuda")[:, None]
        b = torch.arange(Kb, device="cuda")[None, :]
        return (m // 128) * (Kb // 4) * 512 + (b // 4) * 512 + (m % 32) * 16 + (m % 128) // 32 * 4 + b % 4

    def nvfp4(y, dtype):
        H = y.shape[1]
        g = float(s["scale"])
        back = torch.empty(M, H, dtype=dtype, device="cuda")
        codes = torch.zeros(-(-M // 128) * 128 * (H // 16), dtype=torch.uint8, device="cuda")
        for at in range(0, M, 2048):
            b = y[at:at + 2048].to(f64).unflatten(1, (H // 16, 16))
            c = nearest(g * b.abs().amax(2) / 6.0, e4)
            v = e4[c]
            t = b * (g / v)[..., None]
            t = torch.where(v[..., None] == 0, torch.zeros_like(t), t)
            x = (torch.copysign(e2[nearest(t, e2)], t) * v[..., None] / g).flatten(1)
            back[at:at + 2048] = to_e4m3(x) if dtype is E4M3 else x.to(dtype)
            codes[offsets(M, H // 16)[at:at + 2048].reshape(-1)] = c.to(torch.uint8).reshape(-1)
        return back, codes.reshape(-1, H // 16).view(E4M3)

    def mode_outputs(y):
        if case["mode"] == "none":
            return (y,)
        if case["mode"] == "fp8":
            return (to_e4m3(y.to(f64) / float(s["scale"])),)
        return nvfp4(y, E4M3)

    op = case["op"]
    if op == "quantize":
        return nvfp4(s["x"], T)
    if op == "gated":
        H = case["H"]
        y = torch.empty(M, H, dtype=T, device="cuda")
        for at in range(0, M, 4096):
            a, u = s["x"][at:at + 4096].to(f64).split(H, 1)
            if case["act"] == "silu":
                a = a * torch.sigmoid(a)
            else:
                a = 0.5 * a * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (a + 0.044715 * a.pow(3))))
            y[at:at + 4096] = (a * u).to(T)
        return mode_outputs(y)
    if op == "sandwich":
        h, y = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        for at in range(0, M, 4096):
            rows = slice(at, at + 4096)
            z = s["x"][rows].to(f64)
            z = z / (z.pow(2).mean(1, keepdim=True) + EPS).sqrt() * (s["post"].to(f64) + 1.0)
            gate = s["gate_t"]
            if gate is not None:
                z = z * (gate[rows] if gate.dim() == 2 else gate).to(f64)
            h[rows] = (s["residual"][rows].to(f64) + case["res_scale"] * z).to(T)
            z = h[rows].to(f64)
            y[rows] = (z / (z.pow(2).mean(1, keepdim=True) + EPS).sqrt() * (s["pre"].to(f64) + 1.0)).to(T)
        return (h, *mode_outputs(y))

    def matrix(q, sw):
        rows, half = q.shape
        e = torch.cat((e2, -e2))
        v = torch.empty(rows, 2 * half, dtype=f64, device="cuda")
        v[:, 0::2] = e[(q % 16).long()]
        v[:, 1::2] = e[(q // 16).long()]
        sf = sw.reshape(-1)[offsets(rows, half // 8)].to(f64)
        return v * sf.repeat_interleave(16, 1)

    y = torch.mm(matrix(s["aq"], s["asf"]), matrix(s["bq"], s["bsf"]).t()) * float(s["alpha"])
    if case["bias"]:
        y = y + s["bias_t"].to(f64)
    return (y.to(T),)
