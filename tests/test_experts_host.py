"""CPU checks of the operators of a mixture of experts: what their entry points
and their binding refuse, and the layout of the block scales.  Nothing here
reaches a launch."""
import ctypes
import random

import pytest
import torch

from experts_ref import offsets_of, scale_rows, tile_index

P, i64, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float
# Pointers that are never dereferenced
A, B, C, D, E_, G_, H_ = (0x1000000 * i for i in range(1, 8))


@pytest.fixture(scope="module")
def lib():
    from nvfp4_quant_gemma_gb300 import build
    build.build()
    import nvfp4_quant_gemma_gb300 as pkg
    return pkg.load()


def route(lib, **kw):
    a = dict(x=A, stride=8, t=2, M=4, E=8, k=2, ex=B, w=C, o=D, s=E_)
    a.update(kw)
    return lib.gnq_expert_route(P(a["x"]), i64(a["stride"]), a["t"], i64(a["M"]), i64(a["E"]), a["k"], 1, F(1.0), P(a["ex"]),
                                P(a["w"]), P(a["o"]), P(a["s"]), None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=3), 3), (dict(t=-1), 3), (dict(E=0), 2), (dict(E=1025, stride=1025), 2), (dict(k=0), 2), (dict(k=9), 2),
    (dict(k=33, E=64, stride=64), 2), (dict(M=-1), 2), (dict(M=1 << 27, k=16, E=16, stride=16), 2), (dict(M=1 << 28), 2),
    (dict(stride=7), 6), (dict(stride=(1 << 32) + 1), 6), (dict(x=None), 1), (dict(ex=None), 1), (dict(w=None), 1),
    (dict(o=None), 1), (dict(s=None), 1), (dict(M=0, o=None), 1), (dict(x=A + 2), 6), (dict(t=0, x=A + 1), 6),
    (dict(ex=B + 2), 6), (dict(w=C + 1), 6), (dict(o=D + 2), 6), (dict(s=E_ + 2), 6),
    (dict(ex=A + 4), 5), (dict(w=B + 28), 5), (dict(o=E_ - 32), 5), (dict(s=A + 124), 5), (dict(o=A - 32), 5),
    (dict(stride=64, s=A + 3 * 256), 5), (dict(stride=64, ex=A + 3 * 256 - 28), 5),
])
def test_route_refuses(lib, kw, status):
    assert route(lib, **kw) == status


def quantize(lib, **kw):
    a = dict(x=A, stride=64, act=0, o=B, E=2, s=C, e=C + 0x1000, k=2, g=C + 0x2000, gs=1, q=D, bs=E_, R=8, M=4, H=64, t=0)
    a.update(kw)
    return lib.gnq_expert_quantize(P(a["x"]), i64(a["stride"]), a["act"], P(a["o"]), i64(a["E"]), P(a["s"]), P(a["e"]), a["k"],
                                   P(a["g"]), a["gs"], P(a["q"]), P(a["bs"]), i64(a["R"]), i64(a["M"]), i64(a["H"]), a["t"],
                                   None)


ORDERED = dict(s=None, e=None, R=4)


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), 3), (dict(act=3), 4), (dict(gs=2), 4), (dict(E=0), 2), (dict(E=1025), 2), (dict(R=-1), 2), (dict(M=-1), 2),
    (dict(R=1 << 28), 2), (dict(H=0), 2), (dict(H=96, stride=96), 2), (dict(H=65600, stride=65600), 2), (dict(k=0), 2),
    (dict(k=33), 2), (dict(s=None, e=None), 2), (dict(stride=56), 6), (dict(stride=68), 6), (dict(act=1), 6),
    (dict(x=None), 1), (dict(o=None), 1), (dict(g=None), 1), (dict(q=None), 1), (dict(bs=None), 1), (dict(e=None), 1),
    (dict(s=None, R=4), 1), (dict(x=A + 8), 6), (dict(q=D + 8), 6), (dict(bs=E_ + 2), 6), (dict(o=B + 2), 6), (dict(g=C + 2), 6),
    (dict(s=C + 2), 6), (dict(e=C + 2), 6),
    (dict(M=0), 0), (dict(R=0), 0), (dict(ORDERED, M=0, R=0), 0),
    # outputs over what is read, and over each other
    (dict(q=A + 496), 5), (dict(bs=D + 240), 5), (dict(bs=B + 8), 5), (dict(q=C - 240), 5), (dict(q=C + 0x1000), 5),
    (dict(q=C + 0x2000), 5), (dict(bs=A - 1020), 5), (dict(ORDERED, q=A), 5), (dict(ORDERED, bs=C + 0x2004), 5),
])
def test_quantize_refuses(lib, kw, status):
    assert quantize(lib, **kw) == status


def dequantize(lib, **kw):
    a = dict(q=A, bs=B, o=C, E=2, g=D, gs=1, out=E_, R=4, K=64, t=0)
    a.update(kw)
    return lib.gnq_expert_dequantize(P(a["q"]), P(a["bs"]), P(a["o"]), i64(a["E"]), P(a["g"]), a["gs"], P(a["out"]),
                                     i64(a["R"]), i64(a["K"]), a["t"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=4), 3), (dict(gs=-1), 4), (dict(E=0), 2), (dict(E=1025), 2), (dict(R=-1), 2), (dict(K=32), 2), (dict(K=65600), 2),
    (dict(q=None), 1), (dict(bs=None), 1), (dict(o=None), 1), (dict(out=None), 1), (dict(q=A + 8), 6), (dict(out=E_ + 8), 6),
    (dict(bs=B + 2), 6), (dict(o=C + 2), 6), (dict(g=D + 2), 6), (dict(R=0), 0),
    (dict(out=A + 112), 5), (dict(out=B + 1008), 5), (dict(out=C - 496), 5), (dict(out=D), 5),
])
def test_dequantize_refuses(lib, kw, status):
    assert dequantize(lib, **kw) == status


def linear(lib, **kw):
    a = dict(q=A, bs=B, wq=C, wbs=D, al=E_, als=1, b=None, o=E_ + 0x1000, E=2, y=G_, R=4, N=64, K=64, t=0, bt=0)
    a.update(kw)
    return lib.nvfp4_expert_linear(P(a["q"]), P(a["bs"]), P(a["wq"]), P(a["wbs"]), P(a["al"]), a["als"], P(a["b"]), P(a["o"]),
                                   i64(a["E"]), P(a["y"]), i64(a["R"]), i64(a["N"]), i64(a["K"]), a["t"], a["bt"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=3), 3), (dict(b=H_, bt=2), 3), (dict(b=H_, t=0, bt=1), 3), (dict(als=2), 4), (dict(E=0), 2), (dict(E=1025), 2),
    (dict(R=-1), 2), (dict(R=1 << 28), 2), (dict(N=0), 2), (dict(N=1 << 27), 2), (dict(K=0), 2), (dict(K=96), 2),
    (dict(K=65600), 2), (dict(R=0), 0),
    *[(dict([(n, None)]), 1) for n in ("q", "bs", "wq", "wbs", "al", "o", "y")],
    (dict(q=A + 8), 6), (dict(bs=B + 8), 6), (dict(wq=C + 8), 6), (dict(wbs=D + 8), 6), (dict(y=G_ + 8), 6), (dict(al=E_ + 2), 6),
    (dict(o=E_ + 2), 6), (dict(b=H_ + 1), 6),
    (dict(y=A + 112), 5), (dict(y=B + 1008), 5), (dict(y=C + 4080), 5), (dict(y=D + 1008), 5), (dict(y=E_), 5),
    (dict(y=E_ + 0x1000), 5), (dict(y=H_ - 496, b=H_), 5), (dict(y=H_ + 240, b=H_), 5),
])
def test_linear_refuses(lib, kw, status):
    assert linear(lib, **kw) == status


def combine(lib, **kw):
    a = dict(y=A, s=B, w=C, add=None, out=D, R=8, M=4, H=64, k=2, yt=0, ot=0)
    a.update(kw)
    return lib.gnq_expert_combine(P(a["y"]), P(a["s"]), P(a["w"]), P(a["add"]), P(a["out"]), i64(a["R"]), i64(a["M"]),
                                  i64(a["H"]), a["k"], a["yt"], a["ot"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(yt=3), 3), (dict(ot=3), 3), (dict(yt=0, ot=1), 3), (dict(yt=1, ot=2), 3), (dict(R=-1), 2), (dict(M=-1), 2),
    (dict(k=0), 2), (dict(k=33), 2), (dict(H=0), 2), (dict(H=60), 2), (dict(H=65544), 2), (dict(M=0), 0),
    (dict(y=None), 1), (dict(s=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(y=A + 8), 6), (dict(out=D + 8), 6),
    (dict(add=E_ + 8), 6), (dict(s=B + 2), 6), (dict(w=C + 2), 6),
    (dict(out=A + 1008), 5), (dict(out=B - 496), 5), (dict(out=C + 16), 5), (dict(add=E_, out=E_ + 16), 5),
])
def test_combine_refuses(lib, kw, status):
    assert combine(lib, **kw) == status


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def _t(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


def _gnq():
    import nvfp4_quant_gemma_gb300 as gnq
    return gnq


BF, U8, F32 = torch.bfloat16, torch.uint8, torch.float32


@pytest.mark.parametrize("call", [
    lambda g: g.expert_route(_t(4, 8, dtype=F32)[:, ::2], 2),                       # rows that are not dense
    lambda g: g.expert_route(_t(4, 8, dtype=torch.float64), 2),
    lambda g: g.expert_route(_t(8, dtype=F32), 2),
    lambda g: g.expert_route(_t(4, 8, dtype=F32), 9),
    lambda g: g.expert_route(_t(4, 8, dtype=F32), 0),
    lambda g: g.expert_route(_t(4, 8, dtype=F32), 2, out=(_t(4, 2), _t(4, 2, dtype=F32), _t(8), _t(4, 2))),  # short offsets
    lambda g: g.expert_route(_t(4, 8, dtype=F32), 2, out=(_t(4, 2), _t(4, 2), _t(9), _t(4, 2))),             # weights' type
    lambda g: g.expert_route(_t(4, 8, dtype=F32), 2, out=(_t(4, 2), _t(4, 2, dtype=F32), _t(9), _t(4, 2))),  # not on a device
    lambda g: g.expert_quantize(_t(4, 64, dtype=BF), _t(3), _t(2, dtype=F32), slots=_t(4, 2)),
    lambda g: g.expert_quantize(_t(4, 64, dtype=BF), _t(3), _t(2, dtype=F32), slots=_t(4, 2), experts=_t(4, 1)),
    lambda g: g.expert_quantize(_t(4, 64, dtype=BF), _t(3), _t(2, dtype=F32), slots=_t(5, 2), experts=_t(5, 2)),
    lambda g: g.expert_quantize(_t(4, 64, dtype=BF), _t(3), _t(3, dtype=F32), out=(_t(4, 32, dtype=U8), _t(256, 4, dtype=U8))),
    lambda g: g.expert_quantize(_t(4, 64, dtype=BF), _t(3), _t(2, dtype=F32), out=(_t(3, 32, dtype=U8), _t(256, 4, dtype=U8))),
    lambda g: g.expert_quantize(_t(4, 64, dtype=BF), _t(3), _t(2, dtype=F32), out=(_t(4, 32, dtype=U8), _t(128, 4, dtype=U8))),
    lambda g: g.expert_quantize(_t(4, 64, dtype=BF), _t(3), _t(2, dtype=F32), act="relu"),
    lambda g: g.expert_quantize(_t(4, 64, dtype=BF), _t(3, dtype=torch.int64), _t(2, dtype=F32)),
    lambda g: g.expert_quantize(_t(4, 64, dtype=F32), _t(3), _t(2, dtype=F32)),
    lambda g: g.expert_dequantize(_t(4, 32, dtype=U8), _t(128, 4, dtype=U8), _t(3)),             # short scales
    lambda g: g.expert_dequantize(_t(4, 32, dtype=U8), _t(256, 4, dtype=U8), _t(3), out=_t(4, 64)),
    lambda g: g.expert_dequantize(_t(4, 32, dtype=U8), _t(256, 4, dtype=U8), _t(3), out=_t(3, 64, dtype=BF)),
    lambda g: g.nvfp4_expert_linear(_t(4, 32, dtype=U8), _t(256, 4, dtype=U8), _t(3, 8, 32, dtype=U8), _t(384, 4, dtype=U8),
                                    _t(1, dtype=F32), _t(3)),                                     # another count of experts
    lambda g: g.nvfp4_expert_linear(_t(4, 32, dtype=U8), _t(256, 4, dtype=U8), _t(2, 8, 64, dtype=U8), _t(256, 8, dtype=U8),
                                    _t(1, dtype=F32), _t(3)),                                     # another K
    lambda g: g.nvfp4_expert_linear(_t(4, 32, dtype=U8), _t(256, 4, dtype=U8), _t(2, 8, 32, dtype=U8), _t(128, 4, dtype=U8),
                                    _t(1, dtype=F32), _t(3)),                                     # short weight scales
    lambda g: g.nvfp4_expert_linear(_t(4, 32, dtype=U8), _t(256, 4, dtype=U8), _t(2, 8, 32, dtype=U8), _t(256, 4, dtype=U8),
                                    _t(5, dtype=F32), _t(3)),                                     # alpha's count
    lambda g: g.nvfp4_expert_linear(_t(4, 32, dtype=U8), _t(256, 4, dtype=U8), _t(2, 8, 32, dtype=U8), _t(256, 4, dtype=U8),
                                    _t(2, dtype=F32), _t(3), bias=_t(8, dtype=BF)),               # one expert's bias
    lambda g: g.nvfp4_expert_linear(_t(4, 32, dtype=U8), _t(256, 4, dtype=U8), _t(2, 8, 32, dtype=U8), _t(256, 4, dtype=U8),
                                    _t(2, dtype=F32), _t(3)),                                     # not on a device
    lambda g: g.expert_combine(_t(8, 64, dtype=BF), _t(4, 2), _t(4, 2, dtype=F32), out=_t(4, 64, dtype=F32)),
    lambda g: g.expert_combine(_t(8, 64, dtype=BF), _t(4, 2), _t(4, 1, dtype=F32)),
    lambda g: g.expert_combine(_t(8, 64, dtype=BF), _t(4, 2), _t(4, 2, dtype=F32), add=_t(3, 64, dtype=BF)),
    lambda g: g.expert_combine(_t(8, 64, dtype=BF)[:, ::2], _t(4, 2), _t(4, 2, dtype=F32)),
    lambda g: g.expert_combine(_t(8, 64, dtype=BF), _t(8), _t(8, dtype=F32)),
])
def test_the_binding_refuses(call):
    with pytest.raises((ValueError, RuntimeError)):
        call(_gnq())


# ---------------------------------------------------------------------------
# the layout
# ---------------------------------------------------------------------------
def test_scale_tiles_of_experts_never_meet():
    r = random.Random(4)
    for _ in range(200):
        counts = [r.choice((0, 0, 1, 5, 127, 128, 129, 300)) for _ in range(r.randint(1, 40))]
        offsets = offsets_of(counts)
        index = tile_index(offsets, len(counts), 4).reshape(-1)
        assert index.unique().numel() == index.numel()
        assert index.numel() == 0 or int(index.max()) < scale_rows(offsets[-1], len(counts)) * 4
    assert _gnq().expert_scale_rows(300, 7) == scale_rows(300, 7) == (2 + 7) * 128
