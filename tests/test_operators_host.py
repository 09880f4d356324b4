"""CPU checks of the sandwich norm, quantize, dequantize, gated activation and
NVFP4 product: refusals at the C ABI and in the binding, all before any CUDA
call."""
import ctypes

import pytest
import torch

P, i64, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float
A, B, C, D = (P(0x10000 * i) for i in range(1, 5))  # never dereferenced
ODD = P(0x10002)


@pytest.fixture(scope="module")
def lib():
    from nvfp4_quant_gemma_gb300 import build
    build.build()
    import nvfp4_quant_gemma_gb300 as pkg
    return pkg.load()


def sandwich(lib, **kw):
    a = dict(x=A, r=B, ro=None, wp=C, w=C, gate=None, gs=0, scale=C, mode=0, wy=0, q=D, bs=None, y=None, M=4, H=64, dt=0)
    a.update(kw)
    return lib.gemma_sandwich_norm_quant(a["x"], a["r"], a["ro"], a["wp"], a["w"], a["gate"], i64(a["gs"]), F(1.0),
                                         F(1e-6), a["scale"], a["mode"], a["wy"], a["q"], a["bs"], a["y"],
                                         i64(a["M"]), i64(a["H"]), a["dt"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0, x=None), 0), (dict(dt=2), 3), (dict(mode=3), 4), (dict(mode=-2), 4), (dict(M=-1), 2), (dict(H=60), 2),
    (dict(H=0), 2), (dict(mode=1, bs=D, H=96), 2), (dict(mode=2, bs=D, H=48), 2), (dict(H=65544), 2),
    (dict(H=65528), 2),                        # wider than one CTA and not divisible over a cluster
    (dict(x=None), 1), (dict(r=None), 1), (dict(w=None), 1), (dict(q=None), 1), (dict(scale=None), 1),
    (dict(wy=1), 1), (dict(mode=-1), 1), (dict(mode=1), 1), (dict(mode=2, scale=None), 1),
    (dict(r=A), 5), (dict(ro=A), 5), (dict(wy=1, y=A), 5), (dict(wy=1, y=B), 5), (dict(gate=B), 5),
    (dict(ro=D, wy=1, y=D), 5),
    (dict(x=ODD), 6), (dict(ro=ODD), 6), (dict(wp=ODD), 6), (dict(gate=ODD, gs=64), 6), (dict(gate=D, gs=63), 6),
    (dict(gate=D, gs=68), 6), (dict(gate=D, gs=-8), 6),
])
def test_sandwich_refusals(lib, kw, status):
    assert sandwich(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=0, x=None), 0), (dict(mode=-1), 4), (dict(mode=3), 4), (dict(dt=2), 3), (dict(H=60), 2), (dict(M=-1), 2),
    (dict(mode=1, H=96), 2), (dict(stride=56), 6), (dict(stride=68), 6), (dict(x=None), 1), (dict(q=None), 1),
    (dict(scale=None), 1), (dict(mode=1, bs=None), 1), (dict(x=ODD), 6), (dict(q=ODD), 6),
])
def test_quantize_refusals(lib, kw, status):
    a = dict(x=A, stride=128, scale=B, mode=0, q=C, bs=D, M=4, H=64, dt=0)
    a.update(kw)
    assert lib.gnq_quantize(a["x"], i64(a["stride"]), a["scale"], a["mode"], a["q"], a["bs"], i64(a["M"]), i64(a["H"]),
                            a["dt"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=0, x=None), 0), (dict(act=0), 4), (dict(act=3), 4), (dict(mode=3), 4), (dict(mode=-2), 4), (dict(dt=2), 3),
    (dict(stride=120), 6), (dict(stride=132), 6), (dict(mode=-1, y=None), 1), (dict(wy=1, y=A), 5), (dict(x=None), 1),
    (dict(wy=1, y=ODD), 6),
])
def test_gated_refusals(lib, kw, status):
    a = dict(x=A, stride=128, act=1, scale=B, mode=0, wy=0, q=C, bs=D, y=None, M=4, H=64, dt=0)
    a.update(kw)
    assert lib.gated_act_quant(a["x"], i64(a["stride"]), a["act"], a["scale"], a["mode"], a["wy"], a["q"], a["bs"],
                               a["y"], i64(a["M"]), i64(a["H"]), a["dt"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=0, q=None), 0), (dict(ot=4), 3), (dict(ot=-1), 3), (dict(K=96), 2), (dict(K=0), 2), (dict(M=-1), 2),
    (dict(K=65600), 2), (dict(q=None), 1), (dict(bs=None), 1), (dict(out=None), 1), (dict(out=A), 5), (dict(out=ODD), 6),
])
def test_dequantize_refusals(lib, kw, status):
    a = dict(q=A, bs=B, s=C, out=D, M=4, K=64, ot=0)
    a.update(kw)
    assert lib.gnq_nvfp4_dequantize(a["q"], a["bs"], a["s"], a["out"], i64(a["M"]), i64(a["K"]), a["ot"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=0, q=None), 0), (dict(ot=3), 3), (dict(ot=-1), 3), (dict(bias=D, bt=2), 3), (dict(bias=D, bt=1), 3),
    (dict(K=96), 2), (dict(K=65600), 2), (dict(N=0), 2), (dict(M=-1), 2), (dict(q=None), 1), (dict(wsf=None), 1),
    (dict(alpha=None), 1), (dict(y=None), 1), (dict(y=A), 5), (dict(q=ODD), 6), (dict(sf=P(0x10008)), 6), (dict(y=ODD), 6),
])
def test_linear_refusals(lib, kw, status):
    a = dict(q=A, sf=B, wq=C, wsf=C, alpha=B, bias=None, y=D, M=4, N=64, K=64, ot=0, bt=0)
    a.update(kw)
    assert lib.nvfp4_linear(a["q"], a["sf"], a["wq"], a["wsf"], a["alpha"], a["bias"], a["y"], i64(a["M"]), i64(a["N"]),
                            i64(a["K"]), a["ot"], a["bt"], None) == status


def test_linear_status_has_a_text(lib):
    from nvfp4_quant_gemma_gb300 import status_string
    assert "device memory" in status_string(8)


BF = torch.bfloat16


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refusals(lib):
    """Metadata is refused before placement, and placement (host tensors here) before any launch."""
    import nvfp4_quant_gemma_gb300 as gnq
    s = z(1, dtype=torch.float32)

    def refused(fn, *a, match=None, **k):
        with pytest.raises((ValueError, RuntimeError), match=match):
            fn(*a, **k)

    sw = gnq.gemma_sandwich_norm_quant
    x, w = z(4, 64), z(64)
    outs = (z(4, 32, dtype=torch.uint8), z(128, 4, dtype=torch.uint8), None)
    refused(sw, x, z(4, 64), w, w, 1e-6, s, "nvfp4", out=outs, match="CUDA or pinned")
    refused(sw, x.float(), z(4, 64), w, w, 1e-6, s, "nvfp4", out=outs, match="bf16/fp16")
    refused(sw, x, z(4, 56), w, w, 1e-6, s, "nvfp4", out=outs, match="residual holds")
    refused(sw, x, z(4, 64), w[:60], w, 1e-6, s, "nvfp4", out=outs, match="post_weight holds")
    refused(sw, x, z(4, 64), w, w, 1e-6, None, "nvfp4", out=outs, match="scale must be")
    refused(sw, x, z(4, 64), w, w, 1e-6, s, "nvfp4", gate=z(4, 60), out=outs, match="gate must be")
    refused(sw, x, z(4, 64), w, w, 1e-6, s, "nvfp4", residual_out=z(4, 64, dtype=torch.float16), out=outs,
            match="residual_out must be")
    refused(sw, x, z(4, 64), w, w, 1e-6, s, "nvfp4", out=(outs[0], z(64, 4, dtype=torch.uint8), None),
            match="block_scale holds")
    refused(sw, z(64, 4).t(), z(4, 64), w, w, 1e-6, s, "nvfp4", out=outs, match="contiguous")
    refused(gnq.quantize, z(64, 4).t(), s, "nvfp4", out=outs[:2], match="contiguous rows")
    refused(gnq.quantize, x, s, "nvfp4", out=outs[:2], match="CUDA or pinned")
    refused(gnq.quantize, x, s, "nvfp4", out=(z(4, 16, dtype=torch.uint8), outs[1]), match="q holds")
    refused(gnq.gated_act_quant, z(4, 128), s, "nvfp4", act="relu", out=outs, match="act must be")
    refused(gnq.gated_act_quant, z(4, 129), s, "nvfp4", out=outs, match="even number")
    refused(gnq.gated_act_quant, z(4, 128), s, "nvfp4", out=outs, match="CUDA or pinned")
    q, sf = outs[:2]
    refused(gnq.nvfp4_dequantize, q, sf, s, out=z(4, 64, dtype=torch.float64), match="output must be")
    refused(gnq.nvfp4_dequantize, q, sf, s, out=z(4, 32), match="out holds")
    refused(gnq.nvfp4_dequantize, q, sf, s, out=z(4, 64), match="CUDA or pinned")
    lin = gnq.nvfp4_linear
    wq, wsf = z(8, 32, dtype=torch.uint8), z(128, 4, dtype=torch.uint8)
    refused(lin, q, sf, wq, wsf, s, out=z(4, 8), match="CUDA memory")
    refused(lin, q, sf, z(8, 16, dtype=torch.uint8), wsf, s, out=z(4, 8), match="K = 64")
    refused(lin, q, sf[:64], wq, wsf, s, out=z(4, 8), match="block scales holds")
    refused(lin, q, sf, wq, wsf, z(2, dtype=torch.float32), out=z(4, 8), match="alpha must be")
    refused(lin, q, sf, wq, wsf, s, out=z(4, 8, dtype=torch.float64), match="output must be")
    refused(lin, q, sf, wq, wsf, s, bias=z(8, dtype=torch.float16), out=z(4, 8), match="bias must be")
    refused(lin, q, sf, wq, wsf, s, out=z(4, 7), match="out holds")
