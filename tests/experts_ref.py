"""Plain 64-bit forms of the expert router, the quantization by expert, the
products grouped by expert and the weighted combination, and helpers that build
their operands.  Codes come from the oracle's encoders; nothing here calls the
library."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from gnq_testutil import DTYPE_CODE, bits
from operators_ref import E2M1, linear_tolerance, round_up, swizzle_index


def scale_rows(R, E):
    return (R // 128 + E) * 128


def offsets_of(counts):
    return [0] + np.cumsum(counts).tolist()


def tile_index(offsets, E, Kb):
    """(used rows, Kb) byte offsets of the block scales, by the layout's formula."""
    parts = [((offsets[e] // 128 + e) * (Kb // 4) * 512) + swizzle_index(offsets[e + 1] - offsets[e], Kb)
             for e in range(E)]
    return torch.cat(parts)


def route64(logits, k, renormalize, scale):
    """experts, slots, offsets as the definition gives them (a stable sort in
    Python), weights in fp64; logits any real values, -inf and NaN among them."""
    rows = logits.double().cpu().tolist()
    M, E = len(rows), logits.shape[1]
    inf = float("inf")
    experts, weights = [], []
    for r in rows:
        order = sorted(range(E), key=lambda e: (-inf if r[e] != r[e] else -r[e], e))
        # NaN first: their key is below that of +inf only by place
        order = [e for e in order if r[e] != r[e]] + [e for e in order if r[e] == r[e]]
        pick = [e for e in order if not r[e] == -inf][:k]
        if pick:
            v = torch.tensor(r, dtype=torch.float64)
            m = torch.exp(v - v[pick[0]])
            total = m[pick].sum() if renormalize else m.sum()
            weights.append((scale * m[pick] / total).tolist() + [0.0] * (k - len(pick)))
        else:
            weights.append([0.0] * k)
        experts.append(pick + [-1] * (k - len(pick)))
    slots = [[-1] * k for _ in range(M)]
    offsets, at = [0], 0
    where = [[] for _ in range(E)]
    for t, row in enumerate(experts):
        for j, e in enumerate(row):
            if e >= 0:
                where[e].append((t, j))
    for e in range(E):
        for t, j in where[e]:
            slots[t][j] = at
            at += 1
        offsets.append(at)
    i32 = torch.int32
    return (torch.tensor(experts, dtype=i32).reshape(M, k), torch.tensor(weights, dtype=torch.float64).reshape(M, k),
            torch.tensor(offsets, dtype=i32), torch.tensor(slots, dtype=i32).reshape(M, k))


def quantize_rows(y, scales, offsets, dtype):
    """Codes and scale bytes (plain order) of the used rows of a 16-bit matrix in
    expert order, by the oracle."""
    H = y.shape[1]
    codes, sfs = [], []
    for e in range(len(offsets) - 1):
        a, z = offsets[e], offsets[e + 1]
        if a == z:
            continue
        q, bs = oracle.quantize_from_y(bits(y[a:z]), scales[e], 1, DTYPE_CODE[dtype])
        codes.append(q.reshape(z - a, -1))
        sfs.append(bs.reshape(-1)[swizzle_index(z - a, H // 16).numpy()])
    empty = np.zeros((0, H // 2), np.uint8), np.zeros((0, H // 16), np.uint8)
    return (np.concatenate(codes) if codes else empty[0]), (np.concatenate(sfs) if sfs else empty[1])


def random_rows(offsets, R, K, seed, pad=0x7F):
    """Packed codes (R, K/2) and scales in expert order (CPU); every scale byte
    that belongs to no row holds `pad` (0x7F: E4M3's NaN), as do the codes of
    unused rows."""
    E = len(offsets) - 1
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (R, K // 2), generator=g, dtype=torch.uint8)
    sf = torch.full((scale_rows(R, E) * (K // 16),), pad, dtype=torch.uint8)
    codes = torch.randint(0x20, 0x60, (offsets[-1], K // 16), generator=g, dtype=torch.uint8)
    codes[torch.rand(offsets[-1], K // 16, generator=g) < 0.05] = 0
    if offsets[-1]:
        sf[tile_index(offsets, E, K // 16).reshape(-1)] = codes.reshape(-1)
    return q, sf.reshape(-1, K // 16).view(torch.float8_e4m3fn)


def values(q, sf, index):
    """code * block scale in fp64 (CPU) of packed rows whose scale bytes lie at `index`."""
    q, sf = q.cpu(), sf.cpu().contiguous().view(torch.uint8).reshape(-1)
    v = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64)
    v[:, 0::2] = E2M1[(q & 15).long()]
    v[:, 1::2] = E2M1[(q >> 4).long()]
    return v * sf[index].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)


def expert_linear64(q, sf, wq, wsf, alpha, offsets, bias=None):
    """(result, magnitude of the products) of the used rows in fp64."""
    E, N, K = wq.shape[0], wq.shape[1], 2 * wq.shape[2]
    a = values(q[:offsets[-1]], sf, tile_index(offsets, E, K // 16))
    wsf = wsf.cpu().contiguous().view(torch.uint8).reshape(E, round_up(N, 128), K // 16)
    y = torch.zeros(offsets[-1], N, dtype=torch.float64)
    mag = torch.zeros_like(y)
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        if offsets[e] == offsets[e + 1]:
            continue
        w = values(wq[e], wsf[e], swizzle_index(N, K // 16))
        f = float(alpha[e] if len(alpha) > 1 else alpha[0])
        y[r], mag[r] = a[r] @ w.t() * f, a[r].abs() @ w.abs().t() * abs(f)
        if bias is not None:
            y[r] += bias[e].double().cpu()
            mag[r] += bias[e].double().cpu().abs()
    return y, mag


def linear_bound(y, mag, K, dtype):
    """As for the product of one weight."""
    return linear_tolerance(y, mag, K, dtype)
