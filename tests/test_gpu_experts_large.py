"""GPU tests of the operators of a mixture of experts past 2^31 elements: every
index that does not fit 32 bits shows in the last rows, which are held to the
64-bit forms."""
import pytest
import torch

from experts_ref import linear_bound, quantize_rows, route64, scale_rows, values
from gnq_testutil import u8
from operators_ref import assert_within, rounding, swizzle_index

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gnq():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    from nvfp4_quant_gemma_gb300 import build
    build.build()
    import nvfp4_quant_gemma_gb300 as pkg
    pkg.load()
    import oracle
    oracle.build()
    pkg.read_device_error()
    return pkg


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def test_route_far_rows(gnq):
    """Rows 2^17 elements apart: the last logits lie past 2^31."""
    M, E, k, stride = 17000, 96, 4, 1 << 17
    buf = torch.zeros(M * stride, dtype=torch.bfloat16, device="cuda")
    logits = buf.view(M, stride)[:, 40:40 + E]
    v = torch.randn(M, E, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    logits.copy_(v)
    experts, _, offsets, slots = gnq.expert_route(logits, k)
    got = gnq.expert_route(v.cuda(), k)
    assert torch.equal(experts, got[0]) and torch.equal(offsets, got[2]) and torch.equal(slots, got[3])
    e64, _, _, _ = route64(v[-50:], k, True, 1.0)
    assert torch.equal(experts[-50:].cpu(), e64)


def test_rows_past_2_31_elements(gnq):
    """Quantization, the way back and the combination of 2.3e9 elements."""
    T, M, k, H, E = torch.bfloat16, 8800, 8, 32768, 7
    R = M * k
    x = torch.empty(M, H, dtype=T, device="cuda").normal_()
    slots = torch.randperm(R, generator=torch.Generator().manual_seed(2)).reshape(M, k)
    offsets = [0, 20000, 20000, 20001, 33000, 50000, 70000, R]
    bounds = torch.tensor(offsets)
    experts = torch.searchsorted(bounds[1:], slots, right=True)
    scales = [100.0 + 30 * e for e in range(E)]
    s, o = torch.tensor(scales, device="cuda"), bounds.int().cuda()
    sd, ed = slots.int().cuda(), experts.int().cuda()
    q, sf = gnq.expert_quantize(x, o, s, slots=sd, experts=ed)
    back = gnq.expert_dequantize(q, sf, o, s)
    w = torch.rand(M, k, device="cuda")
    out = gnq.expert_combine(back, sd, w)
    torch.cuda.synchronize()
    assert back.numel() > 1 << 31 and gnq.read_device_error() == 0
    rows = torch.tensor([0, 19999, 20000, 20001, 65535, R - 300, R - 1])
    token = torch.empty(R, dtype=torch.int64)
    token[slots.reshape(-1)] = torch.arange(R) // k
    y = x[token[rows].cuda()].cpu()
    flat, got = sf.view(torch.uint8).reshape(-1), back[rows.cuda()].cpu().float()
    for i, r in enumerate(rows.tolist()):
        e = int(torch.searchsorted(bounds[1:], r, right=True))
        codes, sfs = quantize_rows(y[i:i + 1], [scales[e]], [0, 1], "bf16")
        at = ((offsets[e] // 128 + e) * (H // 64) * 512) + swizzle_index(r - offsets[e] + 1, H // 16)[-1]
        assert (u8(q[r]) == codes[0]).all() and (u8(flat[at.cuda()]) == sfs[0]).all()
        v = values(torch.from_numpy(codes), torch.from_numpy(sfs), torch.arange(H // 16)[None])
        f = torch.from_numpy(sfs).view(torch.float8_e4m3fn).float() / scales[e]
        code = (v / torch.from_numpy(sfs).view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)).nan_to_num().float()
        assert torch.equal(got[i], (code * f.repeat_interleave(16, 1))[0].to(T).float())
    t = torch.tensor([0, M // 2, M - 1])
    terms = back[sd[t.cuda()].long()].cpu().double() * w[t.cuda()].cpu().double()[..., None]
    want, mag = terms.sum(1), terms.abs().sum(1)
    err = (k + 1) * 2.0 ** -24 * mag
    assert_within(out[t.cuda()], want, err + rounding(want.abs() + err, T), "out")


@pytest.mark.parametrize("kernel", [1, 2])
def test_linear_past_2_31(gnq, kernel):
    """Codes, weights and results past 2^31 bytes or elements."""
    R, N, K, E = 135000, 16448, 32768, 9
    offsets = [0, 100, 40000, 40000, 60001, 60002, 90000, 100000, 120000, R]
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randint(0, 256, (R, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    sf = torch.randint(0x28, 0x40, (scale_rows(R, E), K // 16), generator=g, dtype=torch.uint8, device="cuda")
    wq = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    wsf = torch.randint(0x28, 0x40, (E, (N + 127) // 128 * 128, K // 16), generator=g, dtype=torch.uint8, device="cuda")
    alpha = torch.tensor([0.001], device="cuda")
    assert q.numel() > 1 << 31 and wq.numel() > 1 << 31 and R * N > 1 << 31
    gnq.set_linear_policy(kernel)
    try:
        y = gnq.nvfp4_expert_linear(q, sf, wq, wsf, alpha, torch.tensor(offsets, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
    finally:
        gnq.set_linear_policy(0)
    assert gnq.read_device_error() == 0
    cols = torch.tensor([0, 127, 5000, N - 70, N - 1])
    for e, rows in ((0, [0, 99]), (3, [40000, 60000]), (4, [60001]), (8, [120000, R - 129, R - 1])):
        first = (offsets[e] // 128 + e) * (K // 64) * 512
        at = torch.stack([first + swizzle_index(r - offsets[e] + 1, K // 16)[-1] for r in rows])
        a = values(q[rows], sf.reshape(-1)[at.cuda()].cpu(), torch.arange(at.numel()).reshape(at.shape))
        wat = swizzle_index(N, K // 16)[cols]
        b = values(wq[e][cols.cuda()], wsf[e].reshape(-1)[wat.cuda()].cpu(), torch.arange(wat.numel()).reshape(wat.shape))
        f = float(alpha.cpu())
        want, mag = a @ b.t() * f, a.abs() @ b.abs().t() * f
        assert_within(y[rows][:, cols.cuda()], want, linear_bound(want, mag, K, torch.bfloat16), f"expert {e}")
