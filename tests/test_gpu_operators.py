"""GPU tests of the sandwich norm, the quantization of a matrix and its way
back, the gated activation and the NVFP4 product, against plain 64-bit forms.

Sixteen-bit results are within the fp32 error bound of their definition plus
one rounding; codes and block scales are the oracle's, bit for bit, for the
GPU's own 16-bit values; bytes around every output, and scale rows behind the
last row, stay as they were."""
import numpy as np
import pytest
import torch

import oracle
from gnq_testutil import DTYPES, u8
from operators_ref import (act64, assert_within, check_codes, linear64, linear_tolerance, norm64, nvfp4_values,
                           random_nvfp4, round_up, rounding, sandwich64)

pytestmark = pytest.mark.gpu

SENT = 0xA5
GUARD = 256
SCALE = {"fp8": 0.05, "nvfp4": 168.0, "mxfp8": 0.0, "none": 0.0}


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


class Guarded:
    """Buffers with sentinel bytes around and inside them."""

    def __init__(self):
        self.bufs = []

    def __call__(self, shape, dtype, shift=0):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        buf = torch.full((n + 2 * GUARD,), SENT, dtype=torch.uint8, device="cuda")
        at = GUARD + shift
        self.bufs.append((buf, at, n))
        return buf[at:at + n].view(dtype).view(shape)

    def outputs(self, M, H, mode, T, y):
        q = bs = None
        if mode in ("fp8", "mxfp8"):
            q = self((M, H), torch.float8_e4m3fn)
        if mode == "nvfp4":
            q, bs = self((M, H // 2), torch.uint8), self((round_up(M, 128), H // 16), torch.float8_e4m3fn)
        if mode == "mxfp8":
            bs = self((M, H // 32), torch.uint8)
        return q, bs, (self((M, H), T) if y or mode == "none" else None)

    def check(self):
        for buf, at, n in self.bufs:
            b = buf.cpu().numpy()
            assert (b[:at] == SENT).all() and (b[at + n:] == SENT).all(), "bytes around an output were written"


def _gpu_scale(v):
    return torch.tensor([v], dtype=torch.float32, device="cuda")


# ---------------------------------------------------------------------------
# sandwich norm
# ---------------------------------------------------------------------------
def _sandwich_inputs(M, H, T, seed, gate):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, H, generator=g)
    r = torch.randn(M, H, generator=g) * 3
    r[:, :: max(1, H // 5)] *= 20
    if M > 2:
        x[1] = 0.0
        r[2] = 0.0
    wp, w = torch.randn(H, generator=g) * 0.3, torch.randn(H, generator=g) * 0.3
    gt = None
    if gate == "channels":
        gt = torch.randn(H, generator=g).to(T).cuda()
    elif gate == "rows":
        gt = torch.tanh(torch.randn(M, H, generator=g)).to(T).cuda()
    elif gate == "strided":
        gt = torch.tanh(torch.randn(M, H + 24, generator=g)).to(T).cuda()[:, 8:8 + H]
    return [t.to(T).cuda() for t in (x, r, wp, w)] + [gt]


def _run_sandwich(gnq, M, H, dtype, mode, gate="none", post=True, scale=1.0, write_y=True, in_place=False, seed=0,
                  shift=0):
    T = DTYPES[dtype]
    x, r, wp, w, gt = _sandwich_inputs(M, H, T, seed, gate)
    if shift:  # 16-byte but not 32-byte aligned activations
        buf = torch.empty(M * H + 16, dtype=T, device="cuda")
        xs = buf[8:8 + M * H].view(M, H)
        xs.copy_(x)
        x = xs
    wp = wp if post else None
    G = Guarded()
    out = G.outputs(M, H, mode, T, write_y)
    r0 = r.clone()
    h = r if in_place else G((M, H), T)
    s = _gpu_scale(SCALE[mode])
    q, bs, y = gnq.gemma_sandwich_norm_quant(x, r, wp, w, 1e-6, s, mode, gate=gt, residual_scale=scale,
                                             residual_out=None if in_place else h, write_y=write_y, out=out)
    torch.cuda.synchronize()
    G.check()
    if not in_place:
        assert torch.equal(r, r0), "the residual was written"
    h64, err = sandwich64(x, r0, wp, gt, scale)
    assert_within(h, h64, err + rounding(h64.abs() + err, T), "h")
    if y is not None:
        y64 = norm64(h, w)
        err = 2.0 ** -17 * y64.abs()
        assert_within(y, y64, err + rounding(y64.abs() + err, T), "y")
        if mode != "none":
            check_codes(oracle, y, q, bs, SCALE[mode], mode, dtype, SENT)
    return h, q, bs, y


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("mode", ["none", "fp8", "nvfp4", "mxfp8"])
@pytest.mark.parametrize("M,H,gate", [(1, 64, "none"), (3, 2048, "channels"), (130, 2112, "rows"),
                                      (300, 5120, "strided"), (200, 8192, "none")])
def test_sandwich(gnq, M, H, gate, mode, dtype):
    _run_sandwich(gnq, M, H, dtype, mode, gate, scale=0.22 if gate == "channels" else 1.0, seed=M + H)


@pytest.mark.parametrize("mode", ["none", "fp8"])
@pytest.mark.parametrize("M,H", [(1, 8), (5, 200), (160, 1032), (2, 8184)])
def test_sandwich_odd_widths(gnq, M, H, mode):
    _run_sandwich(gnq, M, H, "bf16", mode, "rows", seed=M + H)


@pytest.mark.parametrize("mode,H", [("fp8", 16384), ("mxfp8", 65536), ("nvfp4", 20480), ("nvfp4", 65536)])
@pytest.mark.parametrize("post", [True, False])
def test_sandwich_wide_rows_on_a_cluster(gnq, mode, H, post):
    _run_sandwich(gnq, 5, H, "bf16", mode, "channels", post=post, seed=H)


@pytest.mark.parametrize("mode", ["none", "nvfp4"])
def test_sandwich_without_post_norm_and_in_place(gnq, mode):
    a = _run_sandwich(gnq, 140, 1024, "bf16", mode, "channels", post=False, scale=1.5, seed=9)
    b = _run_sandwich(gnq, 140, 1024, "bf16", mode, "channels", post=False, scale=1.5, seed=9, in_place=True)
    for u, v in zip(a, b):
        assert (u is None) == (v is None) and (u is None or torch.equal(u.view(torch.uint8), v.view(torch.uint8)))


def test_sandwich_16_byte_alignment_and_no_y(gnq):
    """Bits do not depend on the alignment of a buffer, nor on whether y is written."""
    ref = _run_sandwich(gnq, 200, 5120, "bf16", "nvfp4", seed=4)
    for kw in (dict(shift=8), dict(write_y=False)):
        got = _run_sandwich(gnq, 200, 5120, "bf16", "nvfp4", seed=4, **kw)
        for u, v in zip(ref[:3], got[:3]):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def test_sandwich_equals_the_single_norm_without_post_norm(gnq):
    """No post-norm, no gate, scale 1: the residual add and norm that the
    package already has (the same h, and codes from the same y up to one
    rounding of y)."""
    T = torch.bfloat16
    x, r, _, w, _ = _sandwich_inputs(64, 2048, T, 3, "none")
    s = _gpu_scale(168.0)
    r2 = r.clone()
    _, _, y2 = gnq.gemma_add_rms_norm_quant(x, r2, w, 1e-6, s, "nvfp4", write_y=True)
    _, _, y = gnq.gemma_sandwich_norm_quant(x, r, None, w, 1e-6, s, "nvfp4", write_y=True)
    assert torch.equal(r, r2)
    assert_within(y, y2, 2 * rounding(y2.double().cpu().abs(), T), "y")


# ---------------------------------------------------------------------------
# quantization of a matrix, and back
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("mode", ["fp8", "nvfp4", "mxfp8"])
@pytest.mark.parametrize("M,H,extra", [(1, 64, 0), (3, 192, 8), (129, 2048, 2048), (257, 5120, 40), (5, 65536, 0)])
def test_quantize(gnq, M, H, extra, mode, dtype):
    T = DTYPES[dtype]
    g = torch.Generator().manual_seed(M + H)
    x = torch.randn(M, H + extra, generator=g) * 2
    x[0, :16] = 0.0
    if M > 1:
        x[1] = 0.0
        x[1, 3] = 1000.0
    x = x.to(T)
    G = Guarded()
    out = G.outputs(M, H, mode, T, False)[:2]
    q, bs = gnq.quantize(x.cuda()[:, :H], _gpu_scale(SCALE[mode]), mode, out=out)
    torch.cuda.synchronize()
    G.check()
    check_codes(oracle, x[:, :H].contiguous(), q, bs, SCALE[mode], mode, dtype, SENT)


@pytest.mark.parametrize("scale", [0.05, 1e-30, 1e30])
def test_quantize_fp8_extreme_scales(gnq, scale):
    x = (torch.randn(33, 512, generator=torch.Generator().manual_seed(2)) * 3).to(torch.bfloat16)
    q, _ = gnq.quantize(x.cuda(), _gpu_scale(scale), "fp8")
    check_codes(oracle, x, q, None, scale, "fp8", "bf16")


@pytest.mark.parametrize("T", [torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn])
@pytest.mark.parametrize("M,K,g", [(1, 64, None), (130, 320, 168.0), (257, 2048, 3.0)])
def test_dequantize(gnq, M, K, g, T):
    """Bit for bit: code * RN(block scale / g) in fp32, one rounding to the type."""
    q, sf = random_nvfp4(M, K, M + K)
    G = Guarded()
    out = G((M, K), T)
    gnq.nvfp4_dequantize(q.cuda(), sf.cuda(), None if g is None else _gpu_scale(g), out=out)
    torch.cuda.synchronize()
    G.check()
    one = nvfp4_values(torch.full_like(q, 0x22), sf).float()                # the block scales
    code = nvfp4_values(q, torch.full_like(sf.view(torch.uint8), 0x38).view(torch.float8_e4m3fn)).float()
    want = code * (one / (1.0 if g is None else g))
    if T is torch.float8_e4m3fn:
        want = want.clamp(-448, 448)
    assert torch.equal(out.cpu().float(), want.to(T).float())


# ---------------------------------------------------------------------------
# gated activation
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("mode", ["none", "fp8", "nvfp4", "mxfp8"])
@pytest.mark.parametrize("M,H,extra", [(1, 64, 0), (5, 448, 16), (130, 2048, 0)])
def test_gated_act(gnq, M, H, extra, mode, dtype, act):
    T = DTYPES[dtype]
    g = torch.Generator().manual_seed(M + H)
    x = torch.randn(M, 2 * H + extra, generator=g) * 2
    x[0, :8] = torch.tensor([0.0, -0.0, 30.0, -30.0, 100.0, -100.0, 1e4, -1e4])
    x = x.to(T)
    G = Guarded()
    out = G.outputs(M, H, mode, T, True)
    q, bs, y = gnq.gated_act_quant(x.cuda()[:, :2 * H], _gpu_scale(SCALE[mode]), mode, act=act, write_y=True, out=out)
    torch.cuda.synchronize()
    G.check()
    y64 = act64(x[:, :2 * H], act)
    # the exponent's argument t carries 2^-22 |t| (|t| <= 88), the fast
    # exponential 104 units of 2^-23, two products and the quotient; a
    # quotient by more than 2^126 may be 0
    gu = (x[:, :H].double() * x[:, H:2 * H].double()).abs()
    err = 2.0 ** -14 * y64.abs() + 2.0 ** -126 * gu
    assert_within(y, y64, err + rounding(y64.abs() + err, T), "y")
    if mode != "none":
        check_codes(oracle, y, q, bs, SCALE[mode], mode, dtype, SENT)
        q2, bs2, y2 = gnq.gated_act_quant(x.cuda()[:, :2 * H], _gpu_scale(SCALE[mode]), mode, act=act)
        assert y2 is None and np.array_equal(u8(q2), u8(q))


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------
def _run_linear(gnq, M, N, K, T, bias=None, seed=0):
    q, sf = random_nvfp4(M, K, seed)
    wq, wsf = random_nvfp4(N, K, seed + 1)
    alpha = 0.0078125 * 1.37 / K ** 0.5
    b = None
    if bias is not None:
        b = (torch.randn(N, generator=torch.Generator().manual_seed(seed)) * 2).to(bias)
    G = Guarded()
    y = G((M, N), T)
    args = [t.cuda() for t in (q, sf, wq, wsf)]
    a = _gpu_scale(alpha)
    gnq.nvfp4_linear(*args, a, bias=None if b is None else b.cuda(), out=y)
    torch.cuda.synchronize()
    G.check()
    assert gnq.read_device_error() == 0
    y64, mag = linear64(q, sf, wq, wsf, float(a.cpu()), b)
    assert_within(y, y64, linear_tolerance(y64, mag, K, T), "y")
    return args, a, y


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 127, 128, 129, 256, 257, 300, 513])
@pytest.mark.parametrize("N,K", [(128, 256), (200, 320)])
def test_linear_rows(gnq, M, N, K):
    _run_linear(gnq, M, N, K, torch.bfloat16, seed=M + N)


@pytest.mark.parametrize("N", [1, 7, 8, 63, 127, 129, 257, 1000])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_linear_columns(gnq, M, N):
    _run_linear(gnq, M, N, 512, torch.bfloat16, bias=torch.bfloat16, seed=M + N)


@pytest.mark.parametrize("K", [64, 128, 192, 256, 448, 1024, 4160, 8192])
@pytest.mark.parametrize("M,N", [(1, 256), (20, 384), (150, 130), (600, 300)])
def test_linear_depths(gnq, M, N, K):
    _run_linear(gnq, M, N, K, torch.float16, bias=torch.float16, seed=K)


@pytest.mark.parametrize("T,bias", [(torch.float32, None), (torch.float32, torch.bfloat16),
                                    (torch.float32, torch.float16), (torch.float16, None)])
@pytest.mark.parametrize("M,N,K", [(9, 640, 2048), (400, 900, 1024)])
def test_linear_types(gnq, M, N, K, T, bias):
    _run_linear(gnq, M, N, K, T, bias=bias, seed=5)


def test_linear_is_deterministic_and_repeats_in_a_graph(gnq):
    for M, N, K in ((3, 512, 4096), (700, 520, 1024)):
        args, a, y = _run_linear(gnq, M, N, K, torch.bfloat16, seed=1)
        out = torch.zeros_like(y)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            gnq.nvfp4_linear(*args, a, out=out)
        s.synchronize()
        assert torch.equal(out, y)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gnq.nvfp4_linear(*args, a, out=out)
        for _ in range(3):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, y)
        a.mul_(2.0)  # alpha is read on the device: a replay sees the new value
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y * 2)


def test_linear_wait_timeout_writes_nothing(gnq):
    """A bounded wait that gives up: the error bit, no output, and the next call is sound."""
    for M in (5, 300):
        q, sf = random_nvfp4(M, 2048, 1)
        wq, wsf = random_nvfp4(384, 2048, 2)
        args = [t.cuda() for t in (q, sf, wq, wsf)]
        y = torch.full((M, 384), 7.0, dtype=torch.bfloat16, device="cuda")
        gnq.read_device_error()
        gnq.inject_wait_timeout(True)
        try:
            gnq.nvfp4_linear(*args, _gpu_scale(1.0), out=y)
            torch.cuda.synchronize()
        finally:
            gnq.inject_wait_timeout(False)
        assert gnq.read_device_error(clear=True) & 1
        assert bool((y == 7.0).all())
        _run_linear(gnq, M, 384, 2048, torch.bfloat16)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def _mlp(gnq, x, r, gate, wp, w, up_w, down_w, g_in, g_mid, alpha_up, alpha_down):
    """Sandwich norm, gate and up products, gated activation, down product,
    and the sandwich norm of the result: the block of a sandwich-norm model."""
    q, bs, _ = gnq.gemma_sandwich_norm_quant(x, r, wp, w, 1e-6, g_in, "nvfp4", gate=gate)
    gu = gnq.nvfp4_linear(q, bs, *up_w, alpha_up)
    q, bs, _ = gnq.gated_act_quant(gu, g_mid, "nvfp4", act="gelu_tanh")
    d = gnq.nvfp4_linear(q, bs, *down_w, alpha_down)
    return gnq.gemma_sandwich_norm_quant(d, r, wp, w, 1e-6, g_in, "nvfp4", write_y=True), gu, d


@pytest.mark.parametrize("M", [1, 37, 300])
def test_mlp_block(gnq, M):
    H, F, T = 512, 1024, torch.bfloat16
    x, r, wp, w, gate = _sandwich_inputs(M, H, T, 11, "channels")
    r0 = r.clone()
    g = torch.Generator().manual_seed(5)
    wu = (torch.randn(2 * F, H, generator=g) * 0.04).to(T)
    wd = (torch.randn(H, F, generator=g) * 0.04).to(T)
    gw = _gpu_scale(12000.0)
    up_w, down_w = gnq.quantize(wu.cuda(), gw, "nvfp4"), gnq.quantize(wd.cuda(), gw, "nvfp4")
    g_in, g_mid = _gpu_scale(168.0), _gpu_scale(400.0)
    au, ad = 1.0 / (g_in * gw), 1.0 / (g_mid * gw)
    (q, bs, y), gu, d = _mlp(gnq, x, r, gate, wp, w, up_w, down_w, g_in, g_mid, au, ad)
    torch.cuda.synchronize()
    assert gnq.read_device_error() == 0

    # the same steps in 64 bits, each from the values the GPU handed on
    r1 = r0.clone()
    q1, bs1, y1 = gnq.gemma_sandwich_norm_quant(x, r1, wp, w, 1e-6, g_in, "nvfp4", gate=gate, write_y=True)
    h64, err = sandwich64(x, r0, wp, gate, 1.0)
    assert_within(r1, h64, err + rounding(h64.abs() + err, T), "first h")
    check_codes(oracle, y1, q1, bs1, 168.0, "nvfp4", "bf16")
    g64, mag = linear64(q1, bs1, *up_w, float(au.cpu()))
    assert_within(gu, g64, linear_tolerance(g64, mag, H, T), "gate and up")
    qa, bsa, ya = gnq.gated_act_quant(gu, g_mid, "nvfp4", act="gelu_tanh", write_y=True)
    check_codes(oracle, ya, qa, bsa, 400.0, "nvfp4", "bf16")
    d64, mag = linear64(qa, bsa, *down_w, float(ad.cpu()))
    assert_within(d, d64, linear_tolerance(d64, mag, F, T), "down")
    h64, err = sandwich64(d, r1, wp, None, 1.0)
    assert_within(r, h64, err + rounding(h64.abs() + err, T), "second h")
    check_codes(oracle, y, q, bs, 168.0, "nvfp4", "bf16")
    # and the whole block is near the unquantized one: an NVFP4 operand is
    # off by at most a quarter of its value or 1/24 of its block's largest
    full = norm64(r1, w) @ wu.double().t()
    a = act64(full, "gelu_tanh")
    ref = a @ wd.double().t()
    assert float((d.double().cpu() - ref).norm() / ref.norm()) < 0.35


def test_mlp_block_in_a_graph_with_and_without_pdl(gnq):
    M, H, F, T = 16, 512, 1024, torch.bfloat16
    x, r, wp, w, gate = _sandwich_inputs(M, H, T, 12, "rows")
    gw, g_in, g_mid = _gpu_scale(12000.0), _gpu_scale(168.0), _gpu_scale(400.0)
    gen = torch.Generator().manual_seed(6)
    up_w = gnq.quantize((torch.randn(2 * F, H, generator=gen) * 0.04).to(T).cuda(), gw, "nvfp4")
    down_w = gnq.quantize((torch.randn(H, F, generator=gen) * 0.04).to(T).cuda(), gw, "nvfp4")
    au, ad = 1.0 / (g_in * gw), 1.0 / (g_mid * gw)
    r0 = r.clone()

    def run():
        for _ in range(3):
            (q, bs, y), _, d = _mlp(gnq, x, r, gate, wp, w, up_w, down_w, g_in, g_mid, au, ad)
        return y, q

    run()
    torch.cuda.synchronize()
    results = []
    for pdl in (True, False):
        gnq.set_pdl(pdl)
        try:
            r.copy_(r0)
            y, q = run()
            torch.cuda.synchronize()
            results.append((r.clone(), y.clone(), q.clone()))
        finally:
            gnq.set_pdl(True)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y, q = run()
    for _ in range(2):
        r.copy_(r0)
        gr.replay()
        torch.cuda.synchronize()
        results.append((r.clone(), y.clone(), q.clone()))
    for other in results[1:]:
        for u, v in zip(results[0], other):
            assert torch.equal(u, v)


def test_empty_batches(gnq):
    T = torch.bfloat16
    e = torch.empty(0, 128, dtype=T, device="cuda")
    w = torch.zeros(128, dtype=T, device="cuda")
    s = _gpu_scale(1.0)
    q, bs, y = gnq.gemma_sandwich_norm_quant(e, e.clone(), w, w, 1e-6, s, "nvfp4", write_y=True)
    assert q.shape == (0, 64) and y.shape == (0, 128)
    q, bs = gnq.quantize(e, s, "nvfp4")
    assert gnq.nvfp4_dequantize(q, bs, s).shape == (0, 128)
    assert gnq.gated_act_quant(e, s, "fp8")[0].shape == (0, 64)
    wq, wsf = gnq.quantize(torch.zeros(32, 128, dtype=T, device="cuda"), s, "nvfp4")
    assert gnq.nvfp4_linear(q, bs, wq, wsf, s).shape == (0, 32)


def test_linear_with_constant_weights(gnq):
    """The weight read before the wait on the preceding grid: the same bits,
    in a chain whose activation the preceding call writes."""
    H, T = 1024, torch.bfloat16
    gw, gx = _gpu_scale(12000.0), _gpu_scale(60.0)
    gen = torch.Generator().manual_seed(7)
    w = gnq.quantize((torch.randn(H, H, generator=gen) * 0.04).to(T).cuda(), gw, "nvfp4")
    alpha = 1.0 / (gx * gw)
    x0 = (torch.randn(24, H, generator=gen) * 2).to(T).cuda()

    def chain():
        x = x0
        for _ in range(4):
            q, bs = gnq.quantize(x, gx, "nvfp4")
            x = gnq.nvfp4_linear(q, bs, *w, alpha)
        torch.cuda.synchronize()
        return x

    want = chain()
    gnq.set_constant_weights(True)
    try:
        for _ in range(5):
            assert torch.equal(chain(), want)
    finally:
        gnq.set_constant_weights(False)


@pytest.mark.parametrize("M,N,K", [(30, 2049, 2048), (100, 1030, 512), (300, 1001, 512), (1500, 2500, 320),
                                   (700, 8200, 192)])
def test_linear_many_tiles(gnq, M, N, K):
    """More tiles than fit at a time, edges inside tiles, rows of y that tile stores cannot take."""
    for T in (torch.bfloat16, torch.float32):
        _run_linear(gnq, M, N, K, T, bias=torch.bfloat16, seed=M)


def test_linear_two_streams_at_a_time(gnq):
    """Calls of several shapes in flight on two streams give what they give alone."""
    shapes = [(3, 2048, 2048), (60, 1024, 4096), (120, 640, 1024), (400, 1024, 1024)]
    calls = [_run_linear(gnq, M, N, K, torch.bfloat16, seed=M) for M, N, K in shapes]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for i in range(24):
        (args, a, y) = calls[(i * 3) % len(calls)]
        with torch.cuda.stream(streams[i % 2]):
            o = torch.empty_like(y)
            gnq.nvfp4_linear(*args, a, out=o)
            outs.append((o, y))
    torch.cuda.synchronize()
    assert all(torch.equal(o, y) for o, y in outs)
    assert gnq.read_device_error() == 0


def test_infinities_and_nan_stay_in_their_rows(gnq):
    """A row that overflows, and NaN scale bytes of one row, reach no other row."""
    q, sf = random_nvfp4(70, 512, 1)
    wq, wsf = random_nvfp4(260, 512, 2)
    clean = gnq.nvfp4_linear(q.cuda(), sf.cuda(), wq.cuda(), wsf.cuda(), _gpu_scale(1.0), dtype=torch.float16)
    bad = sf.view(torch.uint8).clone().reshape(-1)
    from operators_ref import swizzle_index
    bad[swizzle_index(70, 32)[13]] = 0x7F
    bad = bad.reshape(sf.shape).view(torch.float8_e4m3fn)
    y = gnq.nvfp4_linear(q.cuda(), bad.cuda(), wq.cuda(), wsf.cuda(), _gpu_scale(1.0), dtype=torch.float16)
    keep = torch.arange(70, device="cuda") != 13
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isnan(y[13]).all())


# ---------------------------------------------------------------------------
# places, streams, threads, capture
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("mode", ["none", "fp8", "nvfp4", "mxfp8"])
def test_pinned_host_buffers_give_the_bits_of_device_ones(gnq, mode):
    M, H, T = 130, 1024, torch.bfloat16
    x, r, wp, w, gate = _sandwich_inputs(M, H, T, 21, "rows")
    xg = torch.randn(M, 2 * H, generator=torch.Generator().manual_seed(1)).to(T)
    s = _gpu_scale(SCALE[mode])
    pin = lambda t: None if t is None else t.cpu().pin_memory()

    def same(a, b):
        torch.cuda.synchronize()
        for u, v in zip(a, b):
            if u is not None and v is not None and u.dim() > 1:
                n = min(u.numel(), v.numel())
                u, v = u.cpu().view(torch.uint8), v.cpu().view(torch.uint8)
                if mode == "nvfp4" and u.shape[1] == H // 16:  # padding rows of the scales are not written
                    from operators_ref import swizzle_index
                    i = swizzle_index(M, H // 16).reshape(-1)
                    u, v = u.reshape(-1)[i], v.reshape(-1)[i]
                assert torch.equal(u, v) and n > 0

    for post in (wp, None):
        h1, h2 = torch.empty_like(r), pin(r)
        a = gnq.gemma_sandwich_norm_quant(x, r, post, w, 1e-6, s, mode, gate=gate, residual_out=h1, write_y=True)
        b = gnq.gemma_sandwich_norm_quant(pin(x), pin(r), pin(post), pin(w), 1e-6, pin(s), mode, gate=pin(gate),
                                          residual_out=h2, write_y=True)
        assert not b[2].is_cuda
        same((*a, h1), (*b, h2))
    same(gnq.gated_act_quant(xg.cuda(), s, mode, write_y=True), gnq.gated_act_quant(pin(xg), pin(s), mode, write_y=True))
    if mode != "none":
        same(gnq.quantize(x, s, mode), gnq.quantize(pin(x), pin(s), mode))
    if mode == "nvfp4":
        q, bs = gnq.quantize(x, s, mode)
        same((gnq.nvfp4_dequantize(q, bs, s),), (gnq.nvfp4_dequantize(pin(q), pin(bs), pin(s)),))


@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_fp8_extreme_scales(gnq, scale):
    """Scales outside the corrected quotient's range, on the division path."""
    M, H, T = 33, 512, torch.bfloat16
    x, r, wp, w, _ = _sandwich_inputs(M, H, T, 2, "none")
    q, _, y = gnq.gemma_sandwich_norm_quant(x, r, wp, w, 1e-6, _gpu_scale(scale), "fp8", write_y=True)
    check_codes(oracle, y, q, None, scale, "fp8", "bf16")
    q, _, y = gnq.gated_act_quant(x, _gpu_scale(scale), "fp8", act="silu", write_y=True)
    check_codes(oracle, y, q, None, scale, "fp8", "bf16")


def test_gate_forms_agree(gnq):
    """One gate per channel, the same expanded over the rows, and the same
    written out per row; a single row's gate in two dimensions."""
    M, H, T = 200, 2048, torch.bfloat16
    x, r, wp, w, gate = _sandwich_inputs(M, H, T, 8, "channels")
    outs = []
    for g in (gate, gate.expand(M, H), gate.expand(M, H).contiguous()):
        h = torch.empty_like(r)
        y = gnq.gemma_sandwich_norm_quant(x, r, wp, w, 1e-6, None, "none", gate=g, residual_out=h)[2]
        outs.append((h, y))
    for h, y in outs[1:]:
        assert torch.equal(h, outs[0][0]) and torch.equal(y, outs[0][1])
    one = gnq.gemma_sandwich_norm_quant(x[:1], r[:1].clone(), wp, w, 1e-6, None, "none", gate=gate)[2]
    two = gnq.gemma_sandwich_norm_quant(x[:1], r[:1].clone(), wp, w, 1e-6, None, "none", gate=gate[None])[2]
    assert torch.equal(one, two)


def test_linear_deepest_and_of_a_matrix_with_itself(gnq):
    _run_linear(gnq, 5, 130, 65536, torch.bfloat16, seed=3)
    _run_linear(gnq, 400, 300, 65536, torch.float32, seed=4)
    q, sf = random_nvfp4(200, 512, 9)
    q, sf = q.cuda(), sf.cuda()
    y = gnq.nvfp4_linear(q, sf, q, sf, _gpu_scale(0.01), dtype=torch.float32)
    y64, mag = linear64(q, sf, q, sf, float(torch.tensor(0.01)))
    assert_within(y, y64, linear_tolerance(y64, mag, 512, torch.float32), "y")


def test_a_stream_given_and_two_host_threads(gnq):
    """Calls on a stream that is not the current one, from two threads at a time."""
    import threading
    T = torch.bfloat16
    gw = _gpu_scale(300.0)
    work = []
    for i, M in enumerate((7, 300)):
        x = torch.randn(M, 1024, generator=torch.Generator().manual_seed(i)).to(T).cuda()
        w = torch.randn(640, 1024, generator=torch.Generator().manual_seed(9 + i)).to(T).cuda()
        wq = gnq.quantize(w, gw, "nvfp4")
        want = gnq.nvfp4_linear(*gnq.quantize(x, gw, "nvfp4"), *wq, _gpu_scale(1e-5))
        work.append((x, wq, want, torch.cuda.Stream()))
    alpha = _gpu_scale(1e-5)
    torch.cuda.synchronize()
    errors = []

    def run(x, wq, want, stream):
        try:
            outs = gnq.alloc_outputs(*x.shape, "nvfp4", False, x)[:2]
            ys = [torch.empty_like(want) for _ in range(40)]
            stream.wait_stream(torch.cuda.default_stream())
            for y in ys:
                q, sf = gnq.quantize(x, gw, "nvfp4", out=outs, stream=stream)
                gnq.nvfp4_linear(q, sf, *wq, alpha, out=y, stream=stream)
            stream.synchronize()
            if not all(torch.equal(y, want) for y in ys):
                errors.append("results differ")
        except Exception as e:  # noqa: BLE001 - reported by the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=run, args=a) for a in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_first_calls_of_a_process_inside_a_capture():
    """Every operator's first call is captured: what the library asks the
    runtime for on first use is allowed there."""
    import os
    import subprocess
    import sys
    code = """
import torch, nvfp4_quant_gemma_gb300 as gnq
T = torch.bfloat16
dev = torch.device("cuda")
x = torch.randn(40, 512, device=dev).to(T); r = torch.randn(40, 512, device=dev).to(T); w = torch.randn(512, device=dev).to(T)
s = torch.full((1,), 100.0, device=dev); a = torch.full((1,), 1e-4, device=dev)
wq = torch.randint(0, 256, (1024, 256), dtype=torch.uint8, device=dev)
wsf = torch.randint(0x28, 0x50, (1024, 32), dtype=torch.uint8, device=dev)
big = torch.randint(0, 256, (600, 256), dtype=torch.uint8, device=dev)
bsf = torch.randint(0x28, 0x50, (640, 32), dtype=torch.uint8, device=dev)
h = torch.empty_like(r)
torch.cuda.synchronize()

def run():
    q, sf, _ = gnq.gemma_sandwich_norm_quant(x, r, w, w, 1e-6, s, "nvfp4", residual_out=h)
    y = gnq.nvfp4_linear(q, sf, wq, wsf, a)
    q2, sf2, _ = gnq.gated_act_quant(y, s, "nvfp4")
    q3, sf3 = gnq.quantize(x, s, "nvfp4")
    return y, q2, gnq.nvfp4_dequantize(q3, sf3, s), gnq.nvfp4_linear(big, bsf, wq, wsf, a)

g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = run()
g.replay()
torch.cuda.synchronize()
for u, v in zip(got, run()):
    assert torch.equal(u, v)
assert gnq.read_device_error() == 0
print("capture ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=200)
    assert res.returncode == 0 and "capture ok" in res.stdout, res.stderr[-2000:]


@pytest.mark.parametrize("T", [torch.bfloat16, torch.float32])
def test_linear_large_with_unaligned_rows(gnq, T):
    """Rows of y that are not 16-byte aligned in a batch large enough for
    256 x 256 tiles: the bits of the aligned call on the same weight rows,
    some of which are held to the 64-bit form."""
    M, N, K = 4101, 1296, 4096
    q, sf = random_nvfp4(M, K, 1)
    wq, wsf = random_nvfp4(N, K, 2)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    a = _gpu_scale(1e-3)
    args = (q.cuda(), sf.cuda())
    whole = gnq.nvfp4_linear(*args, wq.cuda(), wsf.cuda(), a, bias=bias.cuda(), dtype=T)
    for n in (1290, 1291):
        G = Guarded()
        y = G((M, n), T)
        gnq.nvfp4_linear(*args, wq.cuda()[:n], wsf.cuda(), a, bias=bias.cuda()[:n].contiguous(), out=y)
        torch.cuda.synchronize()
        G.check()
        assert torch.equal(y, whole[:, :n])
    rows = slice(4096, 4101)
    tail = sf.reshape(-1, 128 * K // 16)[32:].reshape(-1, K // 16)
    y64, mag = linear64(q[rows], tail, wq, wsf, float(a.cpu()), bias)
    assert_within(whole[rows], y64, linear_tolerance(y64, mag, K, T), "y")
    assert gnq.read_device_error() == 0


def test_linear_wait_timeout_of_cta_pairs_writes_nothing(gnq):
    """The same failure path in the kernel of large batches, whose CTA pairs wait on one another."""
    M, N, K = 600, 8192, 1024
    q, sf = random_nvfp4(M, K, 1)
    wq, wsf = random_nvfp4(N, K, 2)
    args = [t.cuda() for t in (q, sf, wq, wsf)]
    want = gnq.nvfp4_linear(*args, _gpu_scale(1e-3))
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    gnq.read_device_error()
    gnq.inject_wait_timeout(True)
    try:
        gnq.nvfp4_linear(*args, _gpu_scale(1e-3), out=y)
        torch.cuda.synchronize()
    finally:
        gnq.inject_wait_timeout(False)
    assert gnq.read_device_error(clear=True) & 1
    assert bool((y == 7.0).all())
    assert torch.equal(gnq.nvfp4_linear(*args, _gpu_scale(1e-3)), want)
    assert gnq.read_device_error() == 0


@pytest.mark.parametrize("T,bias", [(torch.bfloat16, torch.bfloat16), (torch.float16, None), (torch.float32, torch.float16)])
@pytest.mark.parametrize("M,N,K", [(600, 8200, 1088), (513, 8184, 1216), (770, 8192, 1280), (1300, 8193, 1152)])
def test_linear_cta_pairs(gnq, M, N, K, T, bias):
    """Shapes whose depth and tile count go to the 256 x 256 tiles of CTA
    pairs (two rounds of them and more), with edges inside tiles of rows,
    columns and K, against the 64-bit form."""
    _run_linear(gnq, M, N, K, T, bias=bias, seed=M)
