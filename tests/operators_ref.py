"""Plain 64-bit forms of the sandwich norm, the gated activation and the NVFP4
product, and helpers that build their operands.  Codes come from the oracle's
encoders; nothing here calls the library."""
from __future__ import annotations

import math

import numpy as np
import torch

from gnq_testutil import DTYPE_CODE, DTYPES, bits, u8  # noqa: F401

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)
MODES = {"fp8": 0, "nvfp4": 1, "mxfp8": 2}
# half a step of a rounding, relative to the value
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# the smallest normal value: below it the step is absolute
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -14, torch.float32: 2.0 ** -126}


def round_up(a, b):
    return (a + b - 1) // b * b


def rounding(v: torch.Tensor, dtype) -> torch.Tensor:
    """The most that one rounding of `v` to `dtype` can move it."""
    return HALF_STEP[dtype] * v.abs().clamp(min=TINY[dtype])


def assert_within(got, want, tol, what):
    got, want = got.double().cpu(), want.double().cpu()
    d = (got - want).abs()
    bad = ~(d <= tol.double().cpu())
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(d[bad].max())}"


def swizzle_index(rows: int, Kb: int) -> torch.Tensor:
    m = torch.arange(rows)[:, None]
    b = torch.arange(Kb)[None, :]
    return (m // 128) * (Kb // 4) * 512 + (b // 4) * 512 + (m % 32) * 16 + (m % 128) // 32 * 4 + b % 4


def nvfp4_values(q: torch.Tensor, sf: torch.Tensor) -> torch.Tensor:
    """code * block scale in fp64 (CPU) of packed codes with swizzled scales."""
    q, sf = q.cpu(), sf.cpu().contiguous().view(torch.uint8).reshape(-1)
    rows, half = q.shape
    v = torch.empty(rows, 2 * half, dtype=torch.float64)
    v[:, 0::2] = E2M1[(q & 15).long()]
    v[:, 1::2] = E2M1[(q >> 4).long()]
    s = sf[swizzle_index(rows, half // 8)].view(torch.float8_e4m3fn).double()
    return v * s.repeat_interleave(16, 1)


def random_nvfp4(rows: int, K: int, seed: int, pad: int = 0x7F):
    """Packed codes, all 16 among them, and swizzled scales of a random matrix
    (CPU); scale rows behind the last row hold `pad` (0x7F: E4M3's NaN)."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
    sf = torch.full((round_up(rows, 128) * (K // 16),), pad, dtype=torch.uint8)
    codes = torch.randint(0x20, 0x60, (rows, K // 16), generator=g, dtype=torch.uint8)
    codes[torch.rand(rows, K // 16, generator=g) < 0.05] = 0        # all-zero blocks
    sf[swizzle_index(rows, K // 16).reshape(-1)] = codes.reshape(-1)
    return q, sf.reshape(-1, K // 16).view(torch.float8_e4m3fn)


def linear64(q, sf, wq, wsf, alpha, bias=None):
    """(result, sum of the products' magnitudes) in fp64."""
    a, w = nvfp4_values(q, sf), nvfp4_values(wq, wsf)
    y = a @ w.t() * alpha
    mag = a.abs() @ w.abs().t() * abs(alpha)
    if bias is not None:
        y = y + bias.double().cpu()
        mag = mag + bias.double().cpu().abs()
    return y, mag


def linear_tolerance(y, mag, K: int, dtype):
    """fp32 sums of K / 64 steps of the tensor core, each adding 64 products
    with at most two units of 2^-23 of the magnitudes summed so far (rounding,
    or truncation on alignment), up to 8 joins of partial sums and the final
    multiply-add; then one rounding to the output type."""
    acc = (2 * (K // 64) + 10) * 2.0 ** -23 * mag
    return acc + rounding(y.abs() + acc, dtype)


def sandwich64(x, residual, w_post, gate, scale):
    """(h before rounding, bound on the fp32 error of it) in fp64."""
    x, r = x.double().cpu(), residual.double().cpu()
    u = x
    if w_post is not None:
        u = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * (1.0 + w_post.double().cpu())
    if gate is not None:
        u = u * gate.double().cpu()
    u = scale * u
    # the sum of squares (at most 64 additions deep), rsqrt, and six products
    return r + u, 2.0 ** -17 * u.abs() + 2.0 ** -23 * (r.abs() + u.abs())


def norm64(h, w):
    h = h.double().cpu()
    return h / torch.sqrt(h.square().mean(-1, keepdim=True) + 1e-6) * (1.0 + w.double().cpu())


def act64(x, act):
    x = x.double().cpu()
    g, u = x[:, : x.shape[1] // 2], x[:, x.shape[1] // 2:]
    if act == "silu":
        a = g * torch.sigmoid(g)
    else:
        # (1 + tanh t) / 2 = sigmoid(2 t); 1 + tanh t itself cancels for t far
        # below 0, where it keeps only 2^-53 absolute
        a = g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))
    return a * u


def check_codes(oracle, y, q, bs, scale, mode, dtype, bs_before=None):
    """Codes and scale bytes, bit for bit, from the 16-bit y they were made of."""
    om = MODES[mode]
    qo, bso = oracle.quantize_from_y(bits(y), scale, om, DTYPE_CODE[dtype])
    M, H = y.shape
    assert np.array_equal(u8(q).reshape(M, -1), qo.reshape(M, -1)), "codes differ"
    if mode == "mxfp8":
        assert np.array_equal(u8(bs), bso.reshape(M, -1)), "scales differ"
    if mode == "nvfp4":
        idx = swizzle_index(M, H // 16).reshape(-1).numpy()
        got, want = u8(bs).reshape(-1), bso.reshape(-1)
        assert np.array_equal(got[idx], want[idx]), "block scales differ"
        if bs_before is not None:  # rows behind the last are left as they were
            rest = np.ones(got.size, bool)
            rest[idx] = False
            assert (got[rest] == bs_before).all(), "padding rows written"
