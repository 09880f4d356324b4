"""GPU tests of the operators around the NVFP4 linear where a call goes wrong
in part, at the ends of a value range, or on a kernel that the size alone would
not choose."""
import contextlib
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
from gnq_testutil import DTYPES
from operators_ref import (act64, assert_within, check_codes, linear64, linear_tolerance, norm64, random_nvfp4, rounding,
                           sandwich64, swizzle_index)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gnq():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    from nvfp4_quant_gemma_gb300 import build
    build.build()
    import nvfp4_quant_gemma_gb300 as pkg
    pkg.load()
    oracle.build()
    return pkg


def _one(v):
    return torch.full((1,), v, dtype=torch.float32, device="cuda")


@pytest.mark.parametrize("T", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cta", [0, 1, 3])
@pytest.mark.parametrize("M", [5, 100])
def test_a_split_product_that_loses_one_part_writes_nothing(gnq, M, cta, T):
    """One CTA of each cluster gives up, its peers do not: the error bit, no
    output from any of them, and the next call is sound.  (384 x 2048 at these
    batches is split over four CTAs.)"""
    q, sf = random_nvfp4(M, 2048, 1)
    wq, wsf = random_nvfp4(384, 2048, 2)
    args = [t.cuda() for t in (q, sf, wq, wsf)]
    y = torch.full((M, 384), 7.0, dtype=T, device="cuda")
    gnq.read_device_error()
    gnq.inject_split_timeout(cta)
    try:
        gnq.nvfp4_linear(*args, _one(1.0), out=y)
        torch.cuda.synchronize()
    finally:
        gnq.inject_split_timeout(-1)
    assert gnq.read_device_error(clear=True) & 1
    assert bool((y == 7.0).all())
    gnq.nvfp4_linear(*args, _one(1e-3), out=y)
    torch.cuda.synchronize()
    assert gnq.read_device_error() == 0
    y64, mag = linear64(q, sf, wq, wsf, float(torch.tensor(1e-3)))
    assert_within(y, y64, linear_tolerance(y64, mag, 2048, T), "y")


def test_outputs_between_the_rows_of_a_strided_input(gnq):
    """What a call writes may lie in the gaps of what it reads: codes, scales
    and y in the columns behind a wide stride."""
    M, H, T = 4, 64, torch.bfloat16
    x = torch.randn(M, 2 * H, generator=torch.Generator().manual_seed(1)).to(T).cuda()
    s = _one(0.05)
    want, _, wy = gnq.gated_act_quant(x, s, "fp8", act="silu", write_y=True)
    arena = torch.zeros(M, 1024, dtype=T, device="cuda")
    arena[:, :2 * H] = x
    q = arena[0, 2 * H:2 * H + M * H // 2].view(torch.uint8).view(M, H)           # right behind row 0
    y = arena[1, 1024 - M * H:].view(M, H)                                        # up to row 2
    gnq.gated_act_quant(arena[:, :2 * H], s, "fp8", act="silu", write_y=True, out=(q, None, y))
    torch.cuda.synchronize()
    assert torch.equal(q, want.view(torch.uint8)) and torch.equal(y, wy) and torch.equal(arena[:, :2 * H], x)
    with pytest.raises(RuntimeError, match="distinct"):
        gnq.gated_act_quant(arena[:, :2 * H], s, "fp8", act="silu", out=(arena[2].view(torch.uint8)[:M * H].view(M, H), None, None))


def _far_gates(T):
    """Gates over the whole range where the activation is not just 0 or the gate."""
    g = torch.cat([torch.linspace(-200, 100, 4096), torch.linspace(-92, -86, 1024), torch.linspace(-13, -8.5, 1024),
                   torch.linspace(-4, 4, 2048)]).to(T)
    return g


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gated_activation_over_the_range_of_the_gate(gnq, dtype, act):
    """The errors that the kernel may have, added up: 2^-22 (power of two) and
    2^-23 (reciprocal), 4 roundings of 2^-24, and those of the exponent t =
    log2(e) g or its cubic form, which the power of two multiplies by |t| ln 2:
    the constant and the product for SiLU (1.25 units of 2^-24: float(log2 e) is
    1.3e-8 off), two constants of up to three roundings and three operations
    for tanh-GELU (6 units).  An act(gate) below 2^-218 may be 0."""
    T = DTYPES[dtype]
    g = _far_gates(T)
    up = [1.0, -0.0078, 61440.0] + ([2.0 ** 100, -1e-30] if dtype == "bf16" else [])
    M, H = len(up), g.numel()
    x = torch.empty(M, 2 * H, dtype=T)
    x[:, :H] = g
    x[:, H:] = torch.tensor(up).to(T)[:, None]
    y = gnq.gated_act_quant(x.cuda(), None, "none", act=act)[2]
    g64, u64 = x[:, :H].double(), x[:, H:].double()
    t = g64.abs() * 1.4427 if act == "silu" else 2.3022 * (g64 + 0.044715 * g64 ** 3).abs()
    y64 = act64(x, act)
    err = (2.0 ** -22 + 2.0 ** -23 + (4 + (1.25 if act == "silu" else 6) * 0.6932 * t) * 2.0 ** -24) * y64.abs()
    err = err + 2.0 ** -218 * u64.abs()
    fits = y64.abs() < torch.finfo(T).max
    assert_within(y.cpu()[fits], y64[fits], (err + rounding(y64.abs() + err, T))[fits], "y")
    assert bool(torch.isinf(y.cpu()[y64.abs() > 1.01 * torch.finfo(T).max]).all())


def test_gated_activation_does_not_depend_on_its_neighbours(gnq):
    """A gate far below 0 in a group does not move the others' bits."""
    T = torch.bfloat16
    x = (torch.randn(64, 1024, generator=torch.Generator().manual_seed(3)) * 3).to(T)
    far = x.clone()
    far[:, 5:512:16] = -88.0
    for act in ("silu", "gelu_tanh"):
        a, b = (gnq.gated_act_quant(v.cuda(), None, "none", act=act)[2].cpu() for v in (x, far))
        keep = torch.ones(512, dtype=torch.bool)
        keep[5::16] = False
        assert torch.equal(a[:, keep], b[:, keep])


# ---------------------------------------------------------------------------
# both kernels of the product on shapes that the choice would give to the other
# ---------------------------------------------------------------------------
@contextlib.contextmanager
def linear_kernel(gnq, kernel):
    gnq.set_linear_policy(kernel)
    try:
        yield
    finally:
        gnq.set_linear_policy(0)


def _product(gnq, M, N, K, T, bias=None, shift=0, seed=0):
    """One product between guard bytes, against 64 bits; the bias starts
    `shift` elements into its buffer."""
    q, sf = random_nvfp4(M, K, seed)
    wq, wsf = random_nvfp4(N, K, seed + 1)
    a = _one(0.0078125 * 1.37 / K ** 0.5)
    b = None
    if bias is not None:
        buf = (torch.randn(N + shift, generator=torch.Generator().manual_seed(seed)) * 2).to(bias).cuda()
        b = buf[shift:]
    size = torch.empty((), dtype=T).element_size()
    raw = torch.full((M * N * size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    y = raw[256:256 + M * N * size].view(T).view(M, N)
    gnq.nvfp4_linear(q.cuda(), sf.cuda(), wq.cuda(), wsf.cuda(), a, bias=b, out=y)
    torch.cuda.synchronize()
    assert bool((raw[:256] == 0xA5).all()) and bool((raw[256 + M * N * size:] == 0xA5).all())
    assert gnq.read_device_error() == 0
    y64, mag = linear64(q, sf, wq, wsf, float(a.cpu()), b)
    assert_within(y, y64, linear_tolerance(y64, mag, K, T), "y")


@pytest.mark.parametrize("M", [1, 65, 128, 129, 257])
@pytest.mark.parametrize("N,K", [(1, 64), (8, 320), (255, 128), (257, 192), (1000, 64), (8193, 320)])
def test_cta_pairs_on_small_and_odd_shapes(gnq, M, N, K):
    """Tiles mostly or (the second CTA of a pair) wholly behind the last token,
    one column, and a K inside the first stage."""
    with linear_kernel(gnq, 2):
        _product(gnq, M, N, K, torch.bfloat16, bias=torch.bfloat16, seed=M + N)
        _product(gnq, M, N, K, torch.float32, bias=torch.float16, seed=M + N)


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("T,bias", [(torch.bfloat16, None), (torch.float16, torch.float16), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("M,N,K", [(1300, 8193, 1152), (300, 1001, 512), (1500, 2500, 320), (700, 8200, 192),
                                   (600, 1024, 512), (600, 8200, 1088), (513, 8184, 1216), (770, 8192, 1280)])
def test_both_kernels_of_the_product(gnq, M, N, K, T, bias, kernel):
    """Each, whichever of the two the call would take by itself."""
    with linear_kernel(gnq, kernel):
        _product(gnq, M, N, K, T, bias=bias, seed=M)


def test_the_choice_between_the_kernels_of_the_product(gnq):
    """Shapes where one of them was measured faster by 15 % or more."""
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("the shapes are those of a device of 152 SMs")
    B, F = torch.bfloat16, torch.float32
    for M, N, K, T in ((300, 5000, 4096, B), (512, 4096, 4096, B), (2048, 2048, 1024, B), (128, 2048, 5120, B),
                       (384, 5000, 4096, B)):
        assert gnq.query_linear(M, N, K, T)[0] == 1, (M, N, K)
    for M, N, K, T in ((8192, 8192, 5120, B), (3420, 1224, 192, F), (16384, 8192, 1024, B)):
        assert gnq.query_linear(M, N, K, T)[0] == 2, (M, N, K)


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("T,bias", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float16)])
@pytest.mark.parametrize("N", [512, 515])
def test_a_bias_off_16_bytes(gnq, kernel, T, bias, N):
    with linear_kernel(gnq, kernel):
        for M in (20, 300):
            for shift in (1, 4):
                _product(gnq, M, N, 512, T, bias=bias, shift=shift, seed=shift)


def test_first_calls_of_both_product_kernels_inside_a_capture():
    """What the library asks the runtime for on a kernel's first use is allowed there."""
    code = """
import torch, nvfp4_quant_gemma_gb300 as gnq
dev = torch.device("cuda")
gen = torch.Generator(device=dev).manual_seed(1)
rnd = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen, dtype=torch.uint8, device=dev)
q, sf, wq, wsf = rnd(0, 256, 600, 256), rnd(0x28, 0x50, 640, 32), rnd(0, 256, 1024, 256), rnd(0x28, 0x50, 1024, 32)
a = torch.full((1,), 1e-4, device=dev)
torch.cuda.synchronize()

def run(T):
    out = []
    for kernel in (2, 1):
        gnq.set_linear_policy(kernel)
        out.append(gnq.nvfp4_linear(q, sf, wq, wsf, a, dtype=T))
    return out

for T in (torch.bfloat16, torch.float16, torch.float32):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run(T)
    g.replay()
    torch.cuda.synchronize()
    for u, v in zip(got, run(T)):
        assert torch.equal(u, v) and bool((u != 0).any())
assert gnq.read_device_error() == 0
print("capture ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=200)
    assert res.returncode == 0 and "capture ok" in res.stdout, res.stderr[-2000:]


# ---------------------------------------------------------------------------
# infinities and NaN, and a scale that the preceding kernel writes
# ---------------------------------------------------------------------------
INF, NAN = float("inf"), float("nan")


def _same_or_near(got, want, tol, what):
    """NaN where the definition has NaN, infinities equal, the rest within tol."""
    got, want = got.double().cpu(), want.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN elsewhere"
    big = torch.isinf(want)
    assert torch.equal(got[big], want[big]), f"{what}: infinities differ"
    rest = ~big & ~torch.isnan(want)
    assert_within(got[rest], want[rest], tol.cpu()[rest], what)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("mode", ["fp8", "nvfp4", "mxfp8"])
def test_quantize_infinities_and_nan(gnq, mode, dtype):
    """Infinities saturate as the oracle's encoders say; a NaN reaches only its
    own block's codes and (FP8) only its own code, which is NaN."""
    T, scale = DTYPES[dtype], {"fp8": 0.05, "nvfp4": 168.0, "mxfp8": 1.0}[mode]
    M, H = 37, 512
    x = (torch.randn(M, H, generator=torch.Generator().manual_seed(4)) * 2).to(T)
    inf = x.clone()
    inf[3, 7], inf[3, 100], inf[5] = INF, -INF, INF
    q, bs = gnq.quantize(inf.cuda(), _one(scale), mode)
    check_codes(oracle, inf, q, bs, scale, mode, dtype)
    nan = x.clone()
    nan[9, 33], nan[9, 300] = NAN, -NAN
    a, abs_ = gnq.quantize(x.cuda(), _one(scale), mode)
    b, bbs = gnq.quantize(nan.cuda(), _one(scale), mode)
    block = {"fp8": 1, "nvfp4": 16, "mxfp8": 32}[mode]
    hit = torch.zeros(M, H // block, dtype=torch.bool)
    hit[9, 33 // block] = hit[9, 300 // block] = True
    per = block // 2 if mode == "nvfp4" else block
    a, b = (t.view(torch.uint8).cpu().reshape(M, H // block, per) for t in (a, b))
    assert torch.equal(a[~hit], b[~hit])
    if mode == "fp8":
        assert bool(((b[hit] & 0x7F) == 0x7F).all())
    if mode == "mxfp8":
        assert torch.equal(abs_.cpu()[~hit], bbs.cpu()[~hit])
    if mode == "nvfp4":
        i = swizzle_index(M, H // 16).reshape(-1)[~hit.reshape(-1)]
        assert torch.equal(abs_.view(torch.uint8).reshape(-1).cpu()[i], bbs.view(torch.uint8).reshape(-1).cpu()[i])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gated_activation_of_infinities_and_nan(gnq, dtype, act):
    T = DTYPES[dtype]
    vals = [0.0, -0.0, 1.0, -1.0, 30.0, -30.0, -88.0, INF, -INF, NAN, 6e4, -6e4]
    g = torch.tensor(vals).repeat_interleave(len(vals))
    u = torch.tensor(vals).repeat(len(vals))
    M, H = 3, g.numel()  # 144: a multiple of 8
    x = torch.cat([g, u]).to(T)[None].repeat(M, 1)
    x[1, :H] = 1.5       # a clean row between
    x[1, H:] = 2.0
    y = gnq.gated_act_quant(x.cuda(), None, "none", act=act)[2]
    y64 = act64(x, act)
    y64 = torch.where(y64.abs() > torch.finfo(T).max * (1 + 2.0 ** -12), torch.copysign(torch.tensor(INF).double(), y64), y64)
    err = 2.0 ** -13 * y64.abs() + 2.0 ** -218 * x[:, H:].double().abs()
    _same_or_near(y, y64, err + rounding(y64.abs() + err, T), "y")


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("M,H", [(12, 256), (600, 2048), (4, 16384)])
def test_sandwich_infinities_and_nan_stay_in_their_rows(gnq, M, H, gate):
    T = torch.bfloat16
    gen = torch.Generator().manual_seed(7)
    x, r, g = (torch.randn(M, H, generator=gen).to(T) for _ in range(3))
    wp, w = ((torch.randn(H, generator=gen) * 0.3).to(T) for _ in range(2))
    bx, br = x.clone(), r.clone()
    bx[1, 9], br[2, 17], bx[3, 40] = INF, -INF, NAN

    def run(a, b):
        h = torch.empty(M, H, dtype=T, device="cuda")
        y = gnq.gemma_sandwich_norm_quant(a.cuda(), b.cuda(), wp.cuda(), w.cuda(), 1e-6, None, "none",
                                          gate=g.cuda() if gate else None, residual_out=h)[2]
        return h.cpu(), y.cpu()

    (h0, y0), (h, y) = run(x, r), run(bx, br)
    clean = torch.ones(M, dtype=torch.bool)
    clean[1:4] = False
    assert torch.equal(h[clean], h0[clean]) and torch.equal(y[clean], y0[clean])
    h64, err = sandwich64(bx, br, wp, g if gate else None, 1.0)
    _same_or_near(h[1:4], h64[1:4], (err + rounding(h64.abs() + err, T))[1:4], "h")
    y64 = norm64(h, w)
    _same_or_near(y[1:4], y64[1:4], (2.0 ** -17 * y64.abs() + rounding(y64.abs(), T))[1:4], "y")


def test_a_scale_written_by_the_preceding_kernel(gnq):
    """A kernel that lets its successor start early and writes the successor's
    scale last (a product with one output): every operator reads the new value."""
    T, M, H = torch.bfloat16, 40, 1024
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(M, 2 * H, generator=gen).to(T).cuda()
    r, w = torch.randn(M, H, generator=gen).to(T).cuda(), (torch.randn(H, generator=gen) * 0.3).to(T).cuda()
    q, sf = (t.cuda() for t in random_nvfp4(1, 4096, 3))
    one = float(gnq.nvfp4_linear(q, sf, q, sf, _one(1.0), dtype=torch.float32))
    alphas = [_one(v / one) for v in (150.0, 90.0, 310.0, 40.0)]
    s = torch.zeros(1, 1, dtype=torch.float32, device="cuda")
    h, xc = torch.empty_like(r), x[:, :H].contiguous()

    def chain():
        out = []
        for a in alphas * 3:
            for call in (lambda: gnq.quantize(x[:, :H], s, "nvfp4")[0], lambda: gnq.quantize(x[:, :H], s, "fp8")[0],
                         lambda: gnq.gated_act_quant(x, s, "nvfp4")[0], lambda: gnq.gated_act_quant(x, s, "fp8")[0],
                         lambda: gnq.gemma_sandwich_norm_quant(xc, r, w, w, 1e-6, s, "nvfp4", residual_out=h)[0],
                         lambda: gnq.gemma_sandwich_norm_quant(xc, r, w, w, 1e-6, s, "fp8", residual_out=h)[0],
                         lambda: gnq.nvfp4_dequantize(q, sf, s)):
                s.fill_(1.0)
                gnq.nvfp4_linear(q, sf, q, sf, a, out=s)
                out.append(call())
        torch.cuda.synchronize()
        return [t.view(torch.uint8) for t in out]

    got = chain()
    gnq.set_pdl(False)
    try:
        want = chain()
    finally:
        gnq.set_pdl(True)
    for i, (u, v) in enumerate(zip(got, want)):
        assert torch.equal(u, v), i
    assert not torch.equal(got[0], got[7])  # another scale, other codes


@pytest.mark.parametrize("scale", [0.05, 100.0, 145.0, 1e4, 2.0 ** 80])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_fp8_of_values_that_overflow_16_bits(gnq, dtype, scale):
    """A y of infinity saturates at 448 / -448 in FP8, at any scale, whichever
    operator made it: the norm (both kernels, one activation and partial sums),
    the sandwich norm, the gated activation, the quantization."""
    T, M, H = DTYPES[dtype], 300, 1024
    gen = torch.Generator().manual_seed(8)
    huge = 6e4 if dtype == "fp16" else 3e38
    x, r = (torch.randn(M, H, generator=gen).to(T).cuda() for _ in range(2))
    w = torch.randn(H, generator=gen) * 0.3
    w[5:37:3], w[40] = huge, -huge
    w = w.to(T).cuda()
    s = _one(scale)

    def check(q, y, some=True):
        assert not some or bool(torch.isinf(y).any())
        check_codes(oracle, y, q, None, scale, "fp8", dtype)

    for kernel in (1, 2):
        gnq.set_launch_policy(kernel)
        try:
            for parts in (x, torch.stack((x, r))):
                q, _, y = gnq.gemma_add_rms_norm_quant_parts(parts, r.clone(), w, 1e-6, s, "fp8", write_y=True)
                check(q, y)
        finally:
            gnq.set_launch_policy()
    q, _, y = gnq.gemma_sandwich_norm_quant(x, r.clone(), None, w, 1e-6, s, "fp8", write_y=True)
    check(q, y)
    g = torch.randn(M, 2 * H, generator=gen)
    g[::7, ::5], g[::7, H::5] = huge, huge * 0.99
    g[1::7, H + 2::5] = -INF
    q, _, y = gnq.gated_act_quant(g.to(T).cuda(), s, "fp8", act="silu", write_y=True)
    check(q, y)
    q, _ = gnq.quantize(y, s, "fp8")
    check(q, y)


def test_sandwich_takes_any_real_number(gnq):
    """eps and the residual scale as a NumPy or a one-element torch value, as the other norms take eps."""
    T = torch.bfloat16
    x, r = (torch.randn(5, 256, generator=torch.Generator().manual_seed(i)).to(T).cuda() for i in (1, 2))
    w = torch.zeros(256, dtype=T, device="cuda")
    run = lambda s, e: gnq.gemma_sandwich_norm_quant(x, r.clone(), w, w, e, None, "none", residual_scale=s)[2]
    want = run(0.5, 2.0 ** -20)
    for s, e in ((np.float32(0.5), np.float32(2.0 ** -20)), (torch.tensor(0.5), torch.tensor(2.0 ** -20))):
        assert torch.equal(run(s, e), want)
    assert torch.equal(run(1, 1e-6), run(1.0, 1e-6))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_activation_rounds_nearly_as_well_as_the_plain_form(gnq, act):
    """fp16 results that are not the exact value's nearest: at most a fifth more
    than of the plain fp32 form, whose exponential and quotient are accurate.
    (An error of d relative moves d / 2^-11 of all results across a border, so
    the count measures the fp32 error.  With one rounding more, the gate times
    the reciprocal before times up, the SiLU has 28 % more.)"""
    wrong, plain_wrong = 0, 0
    for seed in range(4):
        x = torch.randn(4096, 2 * 4096, generator=torch.Generator().manual_seed(seed)).half()
        y = gnq.gated_act_quant(x.cuda(), None, "none", act=act)[2]
        g, u = x.cuda().split(4096, 1)
        gd, ud, gf, uf = g.double(), u.double(), g.float(), u.float()
        if act == "silu":
            exact, plain = gd * torch.sigmoid(gd) * ud, gf / (1.0 + torch.exp(-gf)) * uf
        else:
            c = 2.0 * (2.0 / np.pi) ** 0.5
            exact = gd * torch.sigmoid(c * (gd + 0.044715 * gd ** 3)) * ud
            plain = gf / (1.0 + torch.exp(-c * (gf + 0.044715 * gf * gf * gf))) * uf
        wrong += int((y != exact.half()).sum())
        plain_wrong += int((plain.half() != exact.half()).sum())
    assert wrong <= 1.2 * plain_wrong, (wrong, plain_wrong)
