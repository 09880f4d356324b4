"""The operators past 2^31 elements: offsets of rows, codes, scales and outputs
in 64 bits, against the same rows computed in a small call."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gnq():
    if not torch.cuda.is_available():
        pytest.fail("GPU test run without a CUDA device")
    from nvfp4_quant_gemma_gb300 import build
    build.build()
    import nvfp4_quant_gemma_gb300 as pkg
    pkg.load()
    return pkg


def _sample(M):
    """Whole 128-row blocks (so that block scales keep their places): the ends and around element 2^31 of 8192-wide rows."""
    blocks = sorted({0, 1, (1 << 31) // 8192 // 128 - 1, (1 << 31) // 8192 // 128, M // 128 - 1})
    return blocks


def _one(v):
    return torch.full((1,), v, dtype=torch.float32, device="cuda")


def test_quantize_dequantize_and_gated(gnq):
    M, K = 262144 + 384, 8192
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=g)
    s = _one(200.0)
    q, sf = gnq.quantize(x, s, "nvfp4")
    back = gnq.nvfp4_dequantize(q, sf, s)
    f8, _ = gnq.quantize(x, _one(0.05), "fp8")
    for b in _sample(M):
        rows = slice(128 * b, 128 * b + 128)
        q1, sf1 = gnq.quantize(x[rows], s, "nvfp4")
        assert torch.equal(q[rows], q1), b
        assert torch.equal(sf.view(torch.uint8).view(-1, 128 * K // 16)[b], sf1.view(torch.uint8).view(-1)), b
        assert torch.equal(back[rows], gnq.nvfp4_dequantize(q1, sf1, s)), b
        assert torch.equal(f8[rows].view(torch.uint8), gnq.quantize(x[rows], _one(0.05), "fp8")[0].view(torch.uint8)), b
    del q, sf, back, f8
    gq, gsf, _ = gnq.gated_act_quant(x, s, "nvfp4", act="silu")  # reads past 2^31
    for b in _sample(M):
        rows = slice(128 * b, 128 * b + 128)
        q1, sf1, _ = gnq.gated_act_quant(x[rows], s, "nvfp4", act="silu")
        assert torch.equal(gq[rows], q1), b
        assert torch.equal(gsf.view(torch.uint8).view(-1, 128 * K // 32)[b], sf1.view(torch.uint8).view(-1)), b


def test_sandwich(gnq):
    M, H = 262144 + 384, 8192
    g = torch.Generator(device="cuda").manual_seed(4)
    x, r, gate = (torch.empty(M, H, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    for t in (x, r, gate):
        t.normal_(generator=g)
    wp, w = (torch.randn(H, generator=g, device="cuda").mul_(0.3).to(torch.bfloat16) for _ in range(2))
    s = _one(168.0)
    blocks = _sample(M)
    r0 = {b: r[128 * b:128 * b + 128].clone() for b in blocks}
    q, sf, y = gnq.gemma_sandwich_norm_quant(x, r, wp, w, 1e-6, s, "nvfp4", gate=gate, write_y=True)
    for b in blocks:
        rows = slice(128 * b, 128 * b + 128)
        # 512 rows, so that the small call is launched in the same shape
        four = lambda t: torch.cat((t, t, t, t))
        rr = four(r0[b])
        q1, sf1, y1 = gnq.gemma_sandwich_norm_quant(four(x[rows]), rr, wp, w, 1e-6, s, "nvfp4",
                                                    gate=four(gate[rows]), write_y=True)
        assert torch.equal(r[rows], rr[:128]) and torch.equal(y[rows], y1[:128]) and torch.equal(q[rows], q1[:128]), b
        assert torch.equal(sf.view(torch.uint8).view(-1, 128 * H // 16)[b], sf1.view(torch.uint8).view(-1)[:128 * H // 16]), b


def test_linear(gnq):
    """An output of more than 2^31 values and codes past 2^31 bytes."""
    M, N, K = 262144 + 300, 8200, 16384
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    sf = torch.randint(0x28, 0x50, ((M + 127) // 128 * 128, K // 16), generator=g, device="cuda", dtype=torch.uint8)
    wq = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    wsf = torch.randint(0x28, 0x50, ((N + 127) // 128 * 128, K // 16), generator=g, device="cuda", dtype=torch.uint8)
    a = _one(1e-4)
    y = gnq.nvfp4_linear(q, sf, wq, wsf, a)
    torch.cuda.synchronize()
    assert gnq.read_device_error() == 0
    per = 128 * K // 16
    for b in sorted({0, 1, (1 << 31) // N // 128, (1 << 31) // (K // 2) // 128, M // 256 * 2 - 2, M // 128 - 2}):
        b -= b % 2  # whole tiles of the large call
        n = min(512, M - 128 * b)
        rows = slice(128 * b, 128 * b + n)
        sf1 = sf.view(-1, per)[b:b + (n + 127) // 128].reshape(-1, K // 16)
        y1 = gnq.nvfp4_linear(q[rows], sf1, wq, wsf, a)
        assert torch.equal(y[rows], y1), b
