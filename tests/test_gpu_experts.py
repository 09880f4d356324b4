"""GPU tests of the operators of a mixture of experts, against plain 64-bit
forms: the router, quantization by expert and its way back, the products
grouped by expert, the weighted combination, and a layer of them.

Choices, rows, codes and block scales are equal to the last bit; 16-bit and
32-bit results are within the fp32 error bound of their definition plus one
rounding; bytes around every output, rows behind the last used one and scale
bytes of no row stay as they were."""
import numpy as np
import pytest
import torch

import oracle
from experts_ref import (expert_linear64, linear_bound, offsets_of, quantize_rows, random_rows, route64, scale_rows,
                         tile_index)
from gnq_testutil import DTYPES, u8
from operators_ref import assert_within, random_nvfp4, round_up, rounding
from test_gpu_operators import SENT, Guarded

pytestmark = pytest.mark.gpu

ALL = {**DTYPES, "fp32": torch.float32}


@pytest.fixture(scope="module")
def gnq():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    from nvfp4_quant_gemma_gb300 import build
    build.build()
    import nvfp4_quant_gemma_gb300 as pkg
    pkg.load()
    oracle.build()
    pkg.read_device_error()
    return pkg


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def fp32(v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------
def _check_route(gnq, logits, k, renormalize=True, scale=1.0, x=None):
    M, E = logits.shape
    G = Guarded()
    out = (G((M, k), torch.int32), G((M, k), torch.float32), G((E + 1,), torch.int32), G((M, k), torch.int32))
    experts, weights, offsets, slots = gnq.expert_route(logits.cuda() if x is None else x, k, renormalize=renormalize,
                                                        scale=scale, out=out)
    torch.cuda.synchronize()
    G.check()
    e64, w64, o64, s64 = route64(logits, k, renormalize, scale)
    assert torch.equal(experts.cpu(), e64) and torch.equal(offsets.cpu(), o64) and torch.equal(slots.cpu(), s64)
    # exp: 2 units of 2^-23 and |l_j - l_0| 2^-24 of the rounded difference; the
    # sum: what its terms carry, weighted, and 37 additions; quotient, product
    v = logits.double().cpu()
    d = (v - v.amax(1, keepdim=True)).abs()
    mass = torch.exp(-d)
    d = torch.where(mass > 0, d, torch.zeros_like(d))
    spread = torch.nan_to_num((mass * d).sum(1, keepdim=True) / mass.sum(1, keepdim=True))
    own = torch.nan_to_num(d.gather(1, e64.clamp(min=0).long()))
    assert_within(weights, w64, w64.abs() * 2.0 ** -24 * (own + spread + 8 + 37 + 2) + 2.0 ** -140 * abs(scale), "weights")
    return experts, weights, offsets, slots


def _logits(M, E, dtype, seed, ties=False):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(M, E, generator=g) * 2
    if ties:
        v = torch.randint(-2, 3, (M, E), generator=g).float()
        v = torch.where(v == 0, torch.where(torch.rand(M, E, generator=g) < 0.5, -0.0, 0.0), v)
    return v.to(ALL[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,E,k", [(0, 8, 2), (1, 1, 1), (1, 128, 8), (2, 33, 32), (3, 1024, 32), (64, 60, 4),
                                   (65, 60, 4), (257, 256, 8), (1000, 31, 1), (130, 1000, 7), (5000, 257, 6), (700, 8, 8), (4200, 1, 1), (2200, 1024, 2), (33, 100, 3), (32, 129, 4), (1025, 256, 8),
                                   (9001, 100, 3)])
def test_route(gnq, M, E, k, dtype):
    for ties in (False, True):
        _check_route(gnq, _logits(M, E, dtype, M + E, ties), k, renormalize=not ties, scale=2.5 if ties else 1.0)


@pytest.mark.parametrize("M", [7, 300])
def test_route_masked(gnq, M):
    """Tokens without an expert, with fewer than k, experts that nobody may
    choose, and masks of the type's lowest value, which is a number."""
    v = _logits(M, 48, "bf16", 3)
    v[::5] = -float("inf")
    v[:, 7] = -float("inf")
    v[3, 5:] = -float("inf")
    v[4] = torch.finfo(torch.bfloat16).min
    v[6, 2:] = torch.finfo(torch.bfloat16).min
    for renormalize in (True, False):
        _check_route(gnq, v, 6, renormalize)
    _check_route(gnq, torch.full((M, 5), -float("inf")), 2)


def test_route_nan_and_infinities(gnq):
    v = _logits(70, 40, "fp32", 5)
    clean = gnq.expert_route(v.cuda(), 4)
    v[3, 9] = float("nan")
    v[5, 2] = float("inf")
    v[8, 30], v[8, 31] = float("nan"), -float("nan")
    experts, weights, _, slots = gnq.expert_route(v.cuda(), 4)
    e64, _, _, s64 = route64(v, 4, True, 1.0)
    assert torch.equal(experts.cpu(), e64) and torch.equal(slots.cpu(), s64)
    odd = torch.zeros(70, dtype=torch.bool)
    odd[[3, 5, 8]] = True
    assert bool(torch.isnan(weights.cpu()[odd]).all()) and torch.equal(weights.cpu()[~odd], clean[1].cpu()[~odd])


def test_route_strided_odd_alignment_and_large_values(gnq):
    big = _logits(90, 301, "bf16", 9)
    _check_route(gnq, big[:, 17:218], 5, x=big.cuda()[:, 17:218])
    one = _logits(1, 50, "fp32", 2)
    _check_route(gnq, one * 1e37, 3)
    # a common shift changes nothing but the rounding of the differences
    _check_route(gnq, _logits(40, 64, "fp32", 4) + 1000.0, 8, False)


# ---------------------------------------------------------------------------
# quantization by expert, and back
# ---------------------------------------------------------------------------
COUNTS = {
    "few": [0, 1, 0, 3, 17, 0],
    "tiles": [128, 0, 129, 127, 1, 256, 31],
    "one": [0, 0, 300, 0],
    "single": [5],
    "none": [0, 0, 0],
    "many": [i * 7 % 5 for i in range(1024)],
}


def _fan(counts, k, seed):
    """Slots and experts of M tokens that give the experts these many rows; the
    rows of an expert in shuffled order, some choices dropped."""
    offsets = offsets_of(counts)
    n = offsets[-1]
    M = -(-n // k) + 2
    g = torch.Generator().manual_seed(seed)
    row_expert = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    slots = torch.full((M * k,), -1, dtype=torch.int64)
    slots[torch.randperm(M * k, generator=g)[:n]] = torch.randperm(n, generator=g)
    experts = torch.where(slots >= 0, row_expert[slots.clamp(min=0)] if n else slots, -torch.ones_like(slots))
    return offsets, slots.reshape(M, k), experts.reshape(M, k)


def _check_packed(q, bs, y, scales, offsets, dtype):
    """Codes and scale bytes of the used rows; everything else holds the sentinel."""
    E, H = len(offsets) - 1, y.shape[1]
    codes, sfs = quantize_rows(y, scales, offsets, dtype)
    got, n = u8(q), offsets[-1]
    assert np.array_equal(got[:n], codes), "codes differ"
    assert (got[n:] == SENT).all(), "rows of nobody were written"
    got = u8(bs).reshape(-1)
    idx = tile_index(offsets, E, H // 16).reshape(-1).numpy()
    assert np.array_equal(got[idx], sfs.reshape(-1)), "block scales differ"
    rest = np.ones(got.size, bool)
    rest[idx] = False
    assert (got[rest] == SENT).all(), "scale bytes of no row were written"


def _values(M, H, T, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, H, generator=g) * 2
    if M:
        x[0, :16] = 0.0
        x[M // 2, 3] = 1000.0
    return x.to(T)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("counts,H,k", [("few", 64, 3), ("tiles", 192, 8), ("one", 2048, 1), ("single", 128, 5),
                                        ("none", 64, 2), ("many", 64, 32)])
def test_quantize_fanned_out(gnq, counts, H, k, shared, dtype):
    offsets, slots, experts = _fan(COUNTS[counts], k, 1)
    E, (M, k) = len(offsets) - 1, slots.shape
    x = _values(M, H + 24, DTYPES[dtype], M)
    scales = [168.0] * E if shared else [50.0 + 13.0 * (e % 9) for e in range(E)]
    G = Guarded()
    out = G((M * k, H // 2), torch.uint8), G((scale_rows(M * k, E), H // 16), torch.float8_e4m3fn)
    q, bs = gnq.expert_quantize(x.cuda()[:, 8:8 + H], ints(offsets), fp32(scales[:1] if shared else scales),
                                slots=slots.int().cuda(), experts=experts.int().cuda(), out=out)
    torch.cuda.synchronize()
    G.check()
    y = torch.zeros(offsets[-1], H, dtype=x.dtype)
    t, j = (slots >= 0).nonzero(as_tuple=True)
    y[slots[t, j]] = x[t, 8:8 + H]
    _check_packed(q, bs, y, scales, offsets, dtype)
    assert gnq.read_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", [None, "silu", "gelu_tanh"])
@pytest.mark.parametrize("counts,H", [("few", 64), ("tiles", 448), ("one", 2048), ("none", 64), ("many", 64)])
def test_quantize_in_expert_order(gnq, counts, H, act, dtype):
    offsets = offsets_of(COUNTS[counts])
    E, R = len(offsets) - 1, offsets[-1] + 3
    width = H if act is None else 2 * H
    x = _values(R, width + 8, DTYPES[dtype], R)[:, :width]
    scales = [50.0 + 13.0 * (e % 9) for e in range(E)]
    G = Guarded()
    out = G((R, H // 2), torch.uint8), G((scale_rows(R, E), H // 16), torch.float8_e4m3fn)
    xd = torch.zeros(R, width + 8, dtype=x.dtype, device="cuda")[:, :width].copy_(x)
    q, bs = gnq.expert_quantize(xd, ints(offsets), fp32(scales), act=act, out=out)
    y = x.contiguous() if act is None else gnq.gated_act_quant(xd, None, "none", act=act)[2].cpu()
    torch.cuda.synchronize()
    G.check()
    _check_packed(q, bs, y, scales, offsets, dtype)
    assert gnq.read_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_quantize_extreme_scales(gnq, dtype):
    """Global scales in and outside the range of the tabled quotient, block
    scales of every code: bit for bit the oracle's."""
    scales = [1e-38, 2e-30, 7.9e-31, 0.013, 3.0, 447.3, 1e4, 1.2e30, 1.3e30, 3e38]
    counts = [40] * len(scales)
    offsets = offsets_of(counts)
    R, H = offsets[-1], 256
    g = torch.Generator().manual_seed(8)
    x = (torch.randn(R, H, generator=g) * torch.exp2(torch.randint(-14, 12, (R, H // 16, 1), generator=g).float())
         .expand(R, H // 16, 16).reshape(R, H)).to(DTYPES[dtype])
    G = Guarded()
    bufs = [(G((R, H // 2), torch.uint8), G((scale_rows(R, len(counts)), H // 16), torch.float8_e4m3fn)) for _ in range(2)]
    gnq.expert_quantize(x.cuda(), ints(offsets), fp32(scales), out=bufs[0])
    slots = torch.arange(R).reshape(R, 1)
    experts = torch.repeat_interleave(torch.arange(len(counts)), 40).reshape(R, 1)
    gnq.expert_quantize(x.cuda(), ints(offsets), fp32(scales), slots=slots.int().cuda(), experts=experts.int().cuda(), out=bufs[1])
    torch.cuda.synchronize()
    G.check()
    for q, bs in bufs:
        _check_packed(q, bs, x, fp32(scales).cpu().tolist(), offsets, dtype)


@pytest.mark.parametrize("act", [None, "silu"])
def test_quantize_16_byte_alignment(gnq, act):
    """Rows that are 16-byte but not 32-byte aligned give the same bits."""
    offsets = ints(offsets_of(COUNTS["tiles"]))
    R, W = int(offsets[-1]), 512
    x = _values(R, W, torch.bfloat16, 4).cuda()
    shifted = torch.empty(R * W + 16, dtype=x.dtype, device="cuda")[8:8 + R * W].view(R, W).copy_(x)
    s = fp32([77.0])
    bufs = [(torch.zeros(R, W // (4 if act else 2), dtype=torch.uint8, device="cuda"),
             torch.zeros(scale_rows(R, 7), W // (32 if act else 16), dtype=torch.uint8, device="cuda")) for _ in range(2)]
    for v, out in zip((x, shifted), bufs):
        gnq.expert_quantize(v, offsets, s, act=act, out=out)
    assert torch.equal(bufs[0][0], bufs[1][0]) and torch.equal(bufs[0][1], bufs[1][1])


@pytest.mark.parametrize("T", [torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn])
@pytest.mark.parametrize("counts,K,form", [("few", 64, "each"), ("tiles", 320, "one"), ("many", 64, "none"), ("none", 64, "one")])
def test_dequantize(gnq, counts, K, form, T):
    """Bit for bit: code * RN(block scale / g) in fp32, one rounding to the type."""
    offsets = offsets_of(COUNTS[counts])
    E, n = len(offsets) - 1, offsets[-1]
    R = n + 2
    q, sf = random_rows(offsets, R, K, 3)
    scales = [50.0 + 13.0 * (e % 9) for e in range(E)] if form == "each" else [3.0 if form == "one" else 1.0] * E
    G = Guarded()
    out = G((R, K), T)
    gnq.expert_dequantize(q.cuda(), sf.cuda(), ints(offsets), {"each": fp32(scales), "one": fp32([3.0]), "none": None}[form],
                          out=out)
    torch.cuda.synchronize()
    G.check()
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])
    code = lut[torch.stack((q & 15, q >> 4), -1).long()].reshape(R, K)[:n]
    s = sf.view(torch.uint8).reshape(-1)[tile_index(offsets, E, K // 16)].view(torch.float8_e4m3fn).float()
    g = torch.repeat_interleave(torch.tensor(scales), torch.tensor(COUNTS[counts]))[:, None]
    want = code * (s / g).repeat_interleave(16, 1)
    if T is torch.float8_e4m3fn:
        want = want.clamp(-448, 448)
    assert torch.equal(out.cpu()[:n].float(), want.to(T).float())
    assert (u8(out[n:]) == SENT).all()


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def _operands(counts, N, K, seed, extra=0):
    offsets = offsets_of(counts)
    E = len(counts)
    q, sf = random_rows(offsets, offsets[-1] + extra, K, seed)
    w = [random_nvfp4(N, K, seed + 1 + e % 7) for e in range(E)]
    wq = torch.stack([v[0] for v in w])
    wsf = torch.stack([v[1].view(torch.uint8).reshape(round_up(N, 128), K // 16) for v in w]).view(torch.float8_e4m3fn)
    return offsets, q, sf, wq, wsf


def _run_linear(gnq, counts, N, K, T, bias=None, shared=False, seed=0, extra=2):
    offsets, q, sf, wq, wsf = _operands(counts, N, K, seed, extra)
    E, R = len(counts), offsets[-1] + extra
    alpha = [0.01 * (1 + e % 5) / K ** 0.5 for e in range(1 if shared else E)]
    a = fp32(alpha)
    b = None
    if bias is not None:
        b = (torch.randn(E, N, generator=torch.Generator().manual_seed(seed)) * 2).to(bias)
    G = Guarded()
    y = G((R, N), T)
    args = [t.cuda() for t in (q, sf, wq, wsf)]
    o = ints(offsets)
    gnq.nvfp4_expert_linear(*args, a, o, bias=None if b is None else b.cuda(), out=y)
    torch.cuda.synchronize()
    G.check()
    assert gnq.read_device_error() == 0
    n = offsets[-1]
    y64, mag = expert_linear64(q, sf, wq, wsf, a.cpu().double().tolist(), offsets, b)
    assert_within(y[:n], y64, linear_bound(y64, mag, K, T), "y")
    assert (u8(y[n:]) == SENT).all(), "rows of nobody were written"
    return args, a, o, y


@pytest.mark.parametrize("counts", [[1], [0, 1], [2, 0, 0, 5], [16, 17, 15, 0], [31, 32, 33], [48, 64, 65],
                                    [100, 127, 128, 129, 0, 1], [255, 0, 256, 257, 3], [400, 1, 300]])
@pytest.mark.parametrize("N,K", [(128, 256), (200, 320), (520, 128)])
def test_linear_rows(gnq, counts, N, K):
    _run_linear(gnq, counts, N, K, torch.bfloat16, seed=N)


@pytest.mark.parametrize("N", [1, 7, 8, 63, 127, 129, 257, 1000])
@pytest.mark.parametrize("counts", [[0, 1, 3], [40, 0, 90], [300, 5, 150]])
def test_linear_columns(gnq, counts, N):
    _run_linear(gnq, counts, N, 512, torch.bfloat16, bias=torch.bfloat16, seed=N)


@pytest.mark.parametrize("K", [64, 128, 192, 448, 1024, 4160])
@pytest.mark.parametrize("counts,N", [([1, 1], 256), ([20, 3, 0], 384), ([150, 300], 300)])
def test_linear_depths(gnq, counts, N, K):
    _run_linear(gnq, counts, N, K, torch.float16, bias=torch.float16, seed=K)


@pytest.mark.parametrize("T,bias", [(torch.float32, None), (torch.float32, torch.bfloat16),
                                    (torch.float32, torch.float16), (torch.float16, None)])
@pytest.mark.parametrize("counts,N,K", [([3, 0, 6], 640, 1024), ([200, 170, 0, 30], 901, 512)])
@pytest.mark.parametrize("shared", [False, True])
def test_linear_types(gnq, counts, N, K, T, bias, shared):
    _run_linear(gnq, counts, N, K, T, bias=bias, shared=shared, seed=5)


def test_linear_many_experts_and_tiles(gnq):
    _run_linear(gnq, COUNTS["many"], 136, 128, torch.bfloat16, seed=1)
    _run_linear(gnq, [0] * 1023 + [7], 64, 192, torch.bfloat16, seed=2)
    _run_linear(gnq, [(i * 37) % 90 for i in range(60)], 1000, 192, torch.bfloat16, bias=torch.bfloat16, seed=3)
    _run_linear(gnq, [(i * 53) % 500 for i in range(20)], 1101, 192, torch.float32, seed=4)


@pytest.mark.parametrize("T,bias", [(torch.bfloat16, torch.bfloat16), (torch.float16, None), (torch.float32, torch.float16)])
@pytest.mark.parametrize("counts", [[1], [0, 0], [3, 0, 16, 17], [31, 32, 33, 0, 63, 64, 65], [127, 0, 128, 129, 160],
                                    [255, 256, 257, 7], [700, 1, 513]])
@pytest.mark.parametrize("N,K", [(256, 256), (130, 64), (257, 1088), (1001, 192)])
def test_linear_both_kernels(gnq, counts, N, K, T, bias):
    """Either kernel, whichever would be picked, and the same bits from both."""
    got = []
    for kernel in (1, 2):
        gnq.set_linear_policy(kernel)
        try:
            got.append(_run_linear(gnq, counts, N, K, T, bias=bias, seed=N)[3])
        finally:
            gnq.set_linear_policy(0)
    assert torch.equal(got[0][:sum(counts)], got[1][:sum(counts)])


@pytest.mark.parametrize("counts", [[i * 7 % 5 for i in range(1024)], [450 * (i % 7 == 3) + i * 31 % 70 for i in range(100)],
                                    [0] * 40 + [9000] + [0] * 40 + [5], [40] * 300])
@pytest.mark.parametrize("N,K", [(264, 128), (1100, 64)])
def test_linear_both_kernels_over_many_tiles(gnq, counts, N, K):
    """Each CTA takes several tiles, of experts of very different sizes."""
    got = []
    for kernel in (1, 2):
        gnq.set_linear_policy(kernel)
        try:
            got.append(_run_linear(gnq, counts, N, K, torch.bfloat16, seed=K)[3])
        finally:
            gnq.set_linear_policy(0)
    assert torch.equal(got[0][:sum(counts)], got[1][:sum(counts)])


def test_linear_wait_timeout_in_both_kernels(gnq):
    for kernel in (1, 2):
        for counts in ([3, 0, 2], [700, 0, 600]):
            offsets, q, sf, wq, wsf = _operands(counts, 1024, 1024, 1)
            args = [t.cuda() for t in (q, sf, wq, wsf)]
            y = torch.full((offsets[-1], 1024), 7.0, dtype=torch.bfloat16, device="cuda")
            gnq.read_device_error()
            gnq.set_linear_policy(kernel)
            gnq.inject_wait_timeout(True)
            try:
                gnq.nvfp4_expert_linear(*args, fp32([1.0]), ints(offsets), out=y)
                torch.cuda.synchronize()
            finally:
                gnq.inject_wait_timeout(False)
                gnq.set_linear_policy(0)
            assert gnq.read_device_error(clear=True) & 1
            assert bool((y == 7.0).all())
            _run_linear(gnq, counts, 384, 1024, torch.bfloat16)


def test_linear_wait_timeout_with_many_tiles(gnq):
    """Each CTA still has tiles before it when its waits run out."""
    counts = [40, 0, 500] * 100
    offsets, q, sf, wq, wsf = _operands(counts, 640, 256, 1)
    args = [t.cuda() for t in (q, sf, wq, wsf)]
    for kernel in (1, 2):
        y = torch.full((offsets[-1], 640), 7.0, dtype=torch.bfloat16, device="cuda")
        gnq.read_device_error()
        gnq.set_linear_policy(kernel)
        gnq.inject_wait_timeout(True)
        try:
            gnq.nvfp4_expert_linear(*args, fp32([1.0]), ints(offsets), out=y)
            torch.cuda.synchronize()
        finally:
            gnq.inject_wait_timeout(False)
            gnq.set_linear_policy(0)
        assert gnq.read_device_error(clear=True) & 1
        assert bool((y == 7.0).all())
        _run_linear(gnq, counts[:30], 384, 256, torch.bfloat16)


@pytest.mark.parametrize("N,K", [(136, 64), (256, 1088)])
@pytest.mark.parametrize("counts", [[150, 3] + [0] * 14, [1, 0, 65, 190, 64] + [0] * 20, [0, 63, 129] * 12])
def test_linear_few_rows_but_many_for_one(gnq, counts, N, K):
    """Batches that go to tiles of 64 rows, some of which start inside a scale tile."""
    _run_linear(gnq, counts, N, K, torch.bfloat16, bias=torch.bfloat16, seed=N)


@pytest.mark.parametrize("extra", [0, 200])
def test_linear_without_rows(gnq, extra):
    """No expert has a row: nothing is written."""
    _run_linear(gnq, [0, 0, 0], 256, 128, torch.bfloat16, extra=extra)


def test_linear_deepest(gnq):
    _run_linear(gnq, [5, 0, 130], 130, 65536, torch.float32, seed=3)


def test_linear_nan_stays_in_its_row(gnq):
    """NaN scale bytes of one row, of the padding and of unused rows reach no other row."""
    offsets, q, sf, wq, wsf = _operands([70, 0, 140], 260, 512, 1)
    args = lambda s: (q.cuda(), s.cuda(), wq.cuda(), wsf.cuda(), fp32([0.01]), ints(offsets))
    clean = gnq.nvfp4_expert_linear(*args(sf), dtype=torch.float16)
    bad = sf.view(torch.uint8).clone().reshape(-1)
    bad[tile_index(offsets, 3, 32)[100]] = 0x7F
    y = gnq.nvfp4_expert_linear(*args(bad.reshape(sf.shape).view(torch.float8_e4m3fn)), dtype=torch.float16)
    keep = torch.arange(210, device="cuda") != 100
    assert bool(torch.isfinite(clean.float()).all())
    assert torch.equal(y[keep], clean[keep]) and bool(torch.isnan(y[100]).all())


def test_linear_equals_the_product_of_one_weight(gnq):
    """One expert that owns all rows: the same sums as nvfp4_linear, up to the
    order in which a split adds its parts."""
    for M in (9, 300):
        q, sf = random_nvfp4(M, 1024, 1, pad=0)
        wq, wsf = random_nvfp4(384, 1024, 2)
        a = fp32([0.003])
        one = gnq.nvfp4_linear(q.cuda(), sf.cuda(), wq.cuda(), wsf.cuda(), a, dtype=torch.float32)
        need = scale_rows(M, 1)
        room = torch.zeros(need, 64, dtype=torch.uint8)
        room[:sf.shape[0]] = sf.view(torch.uint8)[:need]
        y = gnq.nvfp4_expert_linear(q.cuda(), room.cuda(), wq[None].cuda(), wsf[None].cuda(), a, ints([0, M]),
                                    dtype=torch.float32)
        _, mag = expert_linear64(q, room, wq[None], wsf[None], [0.003], [0, M])
        assert_within(y, one, 2 * linear_bound(one.double().cpu(), mag, 1024, torch.float32), "y")


def test_linear_wait_timeout_writes_nothing(gnq):
    for counts in ([3, 0, 2], [200, 160], [700, 0, 600]):
        offsets, q, sf, wq, wsf = _operands(counts, 1024, 1024, 1)
        args = [t.cuda() for t in (q, sf, wq, wsf)]
        y = torch.full((offsets[-1], 1024), 7.0, dtype=torch.bfloat16, device="cuda")
        gnq.read_device_error()
        gnq.inject_wait_timeout(True)
        try:
            gnq.nvfp4_expert_linear(*args, fp32([1.0]), ints(offsets), out=y)
            torch.cuda.synchronize()
        finally:
            gnq.inject_wait_timeout(False)
        assert gnq.read_device_error(clear=True) & 1
        assert bool((y == 7.0).all())
        _run_linear(gnq, counts, 384, 1024, torch.bfloat16)


# ---------------------------------------------------------------------------
# combination
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("Y,O", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16"), ("fp32", "fp16")])
@pytest.mark.parametrize("add", ["none", "apart", "in place"])
@pytest.mark.parametrize("M,H,k", [(0, 64, 2), (1, 8, 1), (3, 2048, 8), (130, 1000, 5), (700, 264, 32)])
def test_combine(gnq, M, H, k, add, Y, O):
    g = torch.Generator().manual_seed(M + H)
    R = M * k + 5
    y = torch.randn(R, H, generator=g).to(ALL[Y])
    y[R - 5:] = float("nan")  # rows of nobody
    slots = torch.randperm(M * k, generator=g).reshape(M, k)
    if M:
        slots[::3, 0] = -1
        slots[M // 2] = -7  # a token without rows
    w = torch.rand(M, k, generator=g)
    a = torch.randn(M, H, generator=g).to(ALL[O])
    G = Guarded()
    out = G((M, H), ALL[O])
    if add == "in place":
        out.copy_(a)
    got = gnq.expert_combine(y.cuda(), slots.int().cuda(), w.cuda(), out=out,
                             add={"none": None, "apart": a.cuda(), "in place": out}[add])
    torch.cuda.synchronize()
    G.check()
    assert got is out and gnq.read_device_error() == 0
    rows = y.double()[slots.clamp(min=0)] * (w.double() * (slots >= 0))[..., None]
    want, mag = rows.sum(1), rows.abs().sum(1)
    if add != "none":
        want, mag = want + a.double(), mag + a.double().abs()
    err = (k + 1) * 2.0 ** -24 * mag
    assert_within(out, want, err + rounding(want.abs() + err, ALL[O]), "out")


@pytest.mark.parametrize("k", [2, 9])
def test_combine_infinities_and_nan(gnq, k):
    """An infinite or NaN element reaches its own result alone, with its sign;
    a sum that overflows fp32 is infinite."""
    M, H = 20, 64
    g = torch.Generator().manual_seed(k)
    y = torch.randn(M * k, H, generator=g)
    slots = torch.arange(M * k).reshape(M, k)
    w = torch.rand(M, k, generator=g) + 0.5
    y[0, 3], y[k + 1, 5], y[2 * k, 7] = float("inf"), -float("inf"), float("nan")
    y[3 * k:3 * k + 2, 9] = 3e38
    y[4 * k, 11], y[4 * k + 1, 11] = float("inf"), -float("inf")
    out = gnq.expert_combine(y.cuda(), slots.int().cuda(), w.cuda())
    plain = (y[slots] * w[..., None]).sum(1)
    odd = ~torch.isfinite(plain)
    assert odd.sum() == 5 and torch.equal(torch.isfinite(out.cpu()), ~odd)
    assert out[0, 3] == float("inf") and out[1, 5] == -float("inf") and out[3, 9] == float("inf")
    assert bool(torch.isnan(out[2, 7])) and bool(torch.isnan(out[4, 11]))


# ---------------------------------------------------------------------------
# what the device finds
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("bad", [[0, 5, 3, 9], [0, -4, 4, 9], [0, 3, 6, 1 << 30], [2, 3, 6, 9], [0, 1 << 30, -(1 << 30), 9]])
def test_offsets_that_do_not_ascend_are_reported(gnq, bad):
    """Every access stays inside the buffers (row_bound and the checks of
    expert_from), and the device error word tells."""
    R, N, K = 9, 136, 128
    offsets, q, sf, wq, wsf = _operands([3, 3, 3], N, K, 1)
    G = Guarded()
    o = ints(bad)
    y = G((R, N), torch.bfloat16)
    gnq.read_device_error()
    gnq.nvfp4_expert_linear(q.cuda(), sf.cuda(), wq.cuda(), wsf.cuda(), fp32([1.0]), o, out=y)
    torch.cuda.synchronize()
    if bad[0] != 2:
        assert gnq.read_device_error() & 2 and (u8(y) == SENT).all()
    x = torch.randn(R, K, device="cuda").to(torch.bfloat16)
    out = G((R, K // 2), torch.uint8), G((scale_rows(R, 3), K // 16), torch.float8_e4m3fn)
    gnq.expert_quantize(x, o, fp32([9.0]), out=out)
    gnq.expert_dequantize(*out, o, fp32([9.0]), out=G((R, K), torch.bfloat16))
    torch.cuda.synchronize()
    G.check()
    gnq.read_device_error()


def test_slots_that_name_no_row_are_reported(gnq):
    offsets = ints([0, 4, 6])
    x = torch.randn(3, 64, device="cuda").to(torch.bfloat16)
    for slots, experts in (([[0, 6], [1, 4], [2, 5]], [[0, 1], [0, 1], [0, 1]]),       # behind the last row
                           ([[0, 4], [1, 3], [2, 5]], [[0, 1], [0, 1], [0, 1]]),       # another expert's row
                           ([[0, 4], [1, 5], [2, 3]], [[0, 1], [0, 2], [0, -1]]),      # experts that do not exist
                           ([[0, 4], [1, 5], [2, 1 << 30]], [[0, 1], [0, 1], [0, 1 << 30]])):
        G = Guarded()
        out = G((6, 32), torch.uint8), G((scale_rows(6, 2), 4), torch.uint8)
        gnq.read_device_error()
        gnq.expert_quantize(x, offsets, fp32([9.0]), slots=ints(slots), experts=ints(experts), out=out)
        torch.cuda.synchronize()
        G.check()
        assert gnq.read_device_error() & 2
        rows = {s for t, e in zip(slots, experts) for s, f in zip(t, e) if f in (0, 1) and [0, 4, 6][f] <= s < [0, 4, 6][f + 1]}
        for r in range(6):
            assert (r in rows) != bool((u8(out[0])[r] == SENT).all())
    y = torch.randn(6, 64, device="cuda")
    gnq.read_device_error()
    got = gnq.expert_combine(y, ints([[0, 6], [1, 1 << 30]]), fp32([[1.0, 1.0], [1.0, 1.0]]))
    torch.cuda.synchronize()
    assert gnq.read_device_error() & 2 and torch.equal(got, y[:2])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def _layer(gnq, x, logits, k, w1, w2, s1, s2, a1, a2, shared):
    """A mixture of experts as a block uses it: router, rows to the experts,
    gate and up products, gated activation, down products, weighted sum."""
    experts, weights, offsets, slots = gnq.expert_route(logits, k)
    q, sf = gnq.expert_quantize(x, offsets, s1, slots=slots, experts=experts)
    gu = gnq.nvfp4_expert_linear(q, sf, *w1, a1, offsets)
    q2, sf2 = gnq.expert_quantize(gu, offsets, s2, act="silu")
    d = gnq.nvfp4_expert_linear(q2, sf2, *w2, a2, offsets)
    return gnq.expert_combine(d, slots, weights, add=shared), (experts, weights, offsets, slots, q, sf, gu, q2, sf2, d)


def _layer_inputs(gnq, M, E, H, F, seed, padded=0):
    g = torch.Generator().manual_seed(seed)
    T = torch.bfloat16
    x = torch.randn(M, H, generator=g).to(T).cuda()
    logits = (torch.randn(M, E, generator=g) * 1.5).to(T)
    if padded:
        logits[M - padded:] = -float("inf")
    shared = torch.randn(M, H, generator=g).to(T).cuda()
    gw = fp32([9000.0])

    def weight(N, K):
        parts = [gnq.quantize((torch.randn(N, K, generator=g) * 0.04).to(T).cuda(), gw, "nvfp4") for _ in range(E)]
        return torch.stack([p[0] for p in parts]), torch.stack([p[1].view(torch.uint8) for p in parts])

    s1 = fp32([100.0 + 10 * e for e in range(E)])
    s2 = fp32([300.0 + 20 * e for e in range(E)])
    return x, logits.cuda(), weight(2 * F, H), weight(H, F), s1, s2, 1 / (s1 * gw), 1 / (s2 * gw), shared


@pytest.mark.parametrize("M,E,k,padded", [(1, 16, 4, 0), (37, 6, 2, 5), (300, 10, 3, 0)])
def test_layer(gnq, M, E, k, padded):
    """Every step against its definition, from the values that the GPU handed on."""
    H, F = 512, 384
    x, logits, w1, w2, s1, s2, a1, a2, shared = _layer_inputs(gnq, M, E, H, F, 3, padded)
    out, (experts, weights, offsets, slots, q, sf, gu, q2, sf2, d) = _layer(gnq, x, logits, k, w1, w2, s1, s2, a1, a2, shared)
    torch.cuda.synchronize()
    assert gnq.read_device_error() == 0
    e64, w64, o64, sl64 = route64(logits.cpu(), k, True, 1.0)
    assert torch.equal(experts.cpu(), e64) and torch.equal(slots.cpu(), sl64) and torch.equal(offsets.cpu(), o64)
    o, n = o64.tolist(), int(o64[-1])
    y = torch.zeros(n, H, dtype=torch.bfloat16)
    t, j = (sl64 >= 0).nonzero(as_tuple=True)
    y[sl64[t, j].long()] = x.cpu()[t]

    def packed(q, sf, y, s):
        codes, sfs = quantize_rows(y, s.cpu().tolist(), o, "bf16")
        assert np.array_equal(u8(q)[:n], codes)
        assert np.array_equal(u8(sf).reshape(-1)[tile_index(o, E, y.shape[1] // 16).reshape(-1).numpy()], sfs.reshape(-1))

    packed(q, sf, y, s1)
    r64, mag = expert_linear64(q, sf, *[v.cpu() for v in w1], a1.cpu().double().tolist(), o)
    assert_within(gu[:n], r64, linear_bound(r64, mag, H, torch.bfloat16), "gate and up")
    packed(q2, sf2, gnq.gated_act_quant(gu, None, "none", act="silu")[2].cpu()[:n], s2)
    r64, mag = expert_linear64(q2, sf2, *[v.cpu() for v in w2], a2.cpu().double().tolist(), o)
    assert_within(d[:n], r64, linear_bound(r64, mag, F, torch.bfloat16), "down")
    rows = d.cpu().double()[sl64.clamp(min=0).long()] * (weights.cpu().double() * (sl64 >= 0))[..., None]
    want = rows.sum(1) + shared.cpu().double()
    err = (k + 1) * 2.0 ** -24 * (rows.abs().sum(1) + shared.cpu().double().abs())
    assert_within(out, want, err + rounding(want.abs() + err, torch.bfloat16), "out")


def test_layer_in_a_graph_with_and_without_pdl(gnq):
    """Eager, plain launches and replays give the same bits; a replay routes by
    the logits that it finds."""
    M, E, k, H, F = 70, 12, 3, 512, 384
    inputs = _layer_inputs(gnq, M, E, H, F, 5, 4)
    x, logits = inputs[:2]
    other = logits.flip(0).contiguous()

    def run():
        y = x
        for _ in range(2):  # two layers, the second on what the first wrote
            y, _ = _layer(gnq, y, logits, k, *inputs[2:])
        return y

    first = logits.clone()
    want = {}
    for name, v in (("first", first), ("other", other)):
        logits.copy_(v)
        want[name] = run().clone()
    assert not torch.equal(want["first"], want["other"])
    logits.copy_(first)
    gnq.set_pdl(False)
    try:
        assert torch.equal(run(), want["first"])
    finally:
        gnq.set_pdl(True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for name, v in (("other", other), ("first", first), ("other", other)):
        logits.copy_(v)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want[name])
    assert gnq.read_device_error() == 0


def test_layers_on_two_streams_at_a_time(gnq):
    sets = [(_layer_inputs(gnq, M, 8, 512, 256, M), k) for M, k in ((5, 2), (200, 4), (600, 1))]
    run = lambda s: _layer(gnq, s[0][0], s[0][1], s[1], *s[0][2:])[0]
    want = [run(s) for s in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for i in range(18):
        with torch.cuda.stream(streams[i % 2]):
            outs.append((run(sets[i * 2 % 3]), want[i * 2 % 3]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs) and gnq.read_device_error() == 0


def test_pinned_host_buffers_give_the_bits_of_device_ones(gnq):
    M, E, k, H = 40, 6, 2, 256
    pin = lambda t: t.cpu().pin_memory()
    logits, x = _logits(M, E, "fp32", 1).cuda(), _values(M, H, torch.bfloat16, 2).cuda()
    s = fp32([20.0 + e for e in range(E)])
    a, b = gnq.expert_route(logits, k), gnq.expert_route(pin(logits), k)
    torch.cuda.synchronize()
    assert all(torch.equal(u.cpu(), v) and not v.is_cuda for u, v in zip(a, b))
    qa = gnq.expert_quantize(x, a[2], s, slots=a[3], experts=a[0])
    qb = gnq.expert_quantize(pin(x), b[2], pin(s), slots=b[3], experts=b[0])
    da = gnq.expert_dequantize(*qa, a[2], s)
    db = gnq.expert_dequantize(*qb, b[2], pin(s))
    ca, cb = gnq.expert_combine(da, a[3], a[1]), gnq.expert_combine(db, b[3], b[1])
    torch.cuda.synchronize()
    for u, v in ((qa[0], qb[0]), (da, db), (ca, cb)):
        assert torch.equal(u.cpu(), v) and not v.is_cuda


def test_empty_batches(gnq):
    T = torch.bfloat16
    e = torch.empty(0, 64, dtype=T, device="cuda")
    experts, weights, offsets, slots = gnq.expert_route(torch.empty(0, 4, device="cuda"), 2)
    assert experts.shape == (0, 2) and offsets.tolist() == [0] * 5
    q, sf = gnq.expert_quantize(e, offsets, fp32([1.0]), slots=slots, experts=experts)
    assert q.shape == (0, 32) and gnq.expert_dequantize(q, sf, offsets).shape == (0, 64)
    wq, wsf = torch.zeros(4, 8, 32, dtype=torch.uint8, device="cuda"), torch.zeros(4, 128, 4, dtype=torch.uint8, device="cuda")
    y = gnq.nvfp4_expert_linear(q, sf, wq, wsf, fp32([1.0]), offsets)
    assert y.shape == (0, 8) and gnq.expert_combine(y, slots, weights).shape == (0, 8)
    # tokens, but no rows: the combination is what is added
    none = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    add = torch.randn(3, 8, device="cuda").to(T)
    assert torch.equal(gnq.expert_combine(y, none, torch.ones(3, 2, device="cuda"), add=add), add)


def test_first_calls_of_a_process_inside_a_capture():
    """Every operator's first call is captured: what the library asks the
    runtime for on first use is allowed there."""
    import os
    import subprocess
    import sys
    code = """
import torch, nvfp4_quant_gemma_gb300 as gnq
dev = torch.device("cuda")
sets = []
for M, E, k in ((3, 8, 2), (900, 4, 2)):
    x = torch.randn(M, 256, device=dev).to(torch.bfloat16)
    wq = torch.randint(0, 256, (E, 512, 128), dtype=torch.uint8, device=dev)
    wsf = torch.randint(0x28, 0x50, (E, 512, 16), dtype=torch.uint8, device=dev)
    sets.append((x, torch.randn(M, E, device=dev), k, wq, wsf))
s = torch.full((1,), 100.0, device=dev)
torch.cuda.synchronize()

def run():
    got = []
    for x, logits, k, wq, wsf in sets:
        e, w, o, sl = gnq.expert_route(logits, k)
        q, sf = gnq.expert_quantize(x, o, s, slots=sl, experts=e)
        y = gnq.nvfp4_expert_linear(q, sf, wq, wsf, s, o)
        q2, sf2 = gnq.expert_quantize(y, o, s, act="silu")
        got += [e, w, o, sl, y, q2, gnq.expert_dequantize(q2, sf2, o, s), gnq.expert_combine(y, sl, w)]
    return got

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
