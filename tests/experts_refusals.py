"""Calls of the expert operators that their binding refuses, with the words of
the refusal: the same table for tensors that are on no device (the argument
check comes before that of the place) and for device tensors."""
import torch

BF, F16, U8, F32, I32, I64 = torch.bfloat16, torch.float16, torch.uint8, torch.float32, torch.int32, torch.int64


def calls(t):
    """(name, call, words of the refusal); t(*shape, dtype) makes a tensor."""
    route_out = lambda **kw: tuple({**dict(experts=t(4, 2), weights=t(4, 2, dtype=F32), offsets=t(9), slots=t(4, 2)), **kw}.values())

    def route(g, logits=None, k=2, **kw):
        return g.expert_route(t(4, 8, dtype=F32) if logits is None else logits, k, out=route_out(**kw))

    def quantize(g, x=None, offsets=None, scale=None, q=None, sf=None, fan=False, **kw):
        rows = 8 if fan else 4
        args = dict(slots=t(4, 2), experts=t(4, 2)) if fan else {}
        return g.expert_quantize(t(4, 64, dtype=BF) if x is None else x, t(3) if offsets is None else offsets,
                                 t(2, dtype=F32) if scale is None else scale,
                                 out=(t(rows, 32, dtype=U8) if q is None else q, t(256, 4, dtype=U8) if sf is None else sf),
                                 **{**args, **kw})

    def dequantize(g, q=None, sf=None, offsets=None, scale=None, out=None, **kw):
        return g.expert_dequantize(t(4, 32, dtype=U8) if q is None else q, t(256, 4, dtype=U8) if sf is None else sf,
                                   t(3) if offsets is None else offsets, scale, out=t(4, 64, dtype=BF) if out is None else out, **kw)

    def linear(g, q=None, sf=None, wq=None, wsf=None, alpha=None, offsets=None, out=None, **kw):
        return g.nvfp4_expert_linear(t(4, 32, dtype=U8) if q is None else q, t(256, 4, dtype=U8) if sf is None else sf,
                                     t(2, 8, 32, dtype=U8) if wq is None else wq,
                                     t(2, 128, 4, dtype=U8) if wsf is None else wsf,
                                     t(2, dtype=F32) if alpha is None else alpha, t(3) if offsets is None else offsets,
                                     out=t(4, 8, dtype=BF) if out is None else out, **kw)

    def combine(g, y=None, slots=None, weights=None, out=None, **kw):
        return g.expert_combine(t(8, 64, dtype=BF) if y is None else y, t(4, 2) if slots is None else slots,
                                t(4, 2, dtype=F32) if weights is None else weights,
                                out=t(4, 64, dtype=BF) if out is None else out, **kw)

    return [
        # what the kernels index as matrices
        ("combine: weights of more columns", lambda g: combine(g, weights=t(4, 3, dtype=F32)), r"weights must be \(4, 2\)"),
        ("combine: weights of as many values", lambda g: combine(g, weights=t(2, 4, dtype=F32)), r"weights must be \(4, 2\)"),
        ("combine: flat weights, too many", lambda g: combine(g, weights=t(9, dtype=F32)), r"weights must be \(4, 2\)"),
        ("combine: a wider addend", lambda g: combine(g, add=t(4, 72, dtype=BF)), r"add must be \(4, 64\)"),
        ("combine: an addend of as many values", lambda g: combine(g, add=t(8, 32, dtype=BF)), r"add must be \(4, 64\)"),
        ("linear: a padded bias", lambda g: linear(g, bias=t(2, 16, dtype=BF)), r"bias must be \(2, 8\)"),
        ("linear: a bias of as many values", lambda g: linear(g, bias=t(8, 2, dtype=BF)), r"bias must be \(2, 8\)"),
        ("linear: a padded bias, fp32 result", lambda g: linear(g, out=t(4, 8, dtype=F32), bias=t(2, 16, dtype=F16)),
         r"bias must be \(2, 8\)"),
        ("linear: weight scales of more rows", lambda g: linear(g, wsf=t(2, 256, 4, dtype=U8)),
         r"block scales must be \(2, 128, 4\)"),
        ("linear: weight scales of more columns", lambda g: linear(g, wsf=t(2, 128, 8, dtype=U8)),
         r"block scales must be \(2, 128, 4\)"),
        ("linear: flat weight scales, too many", lambda g: linear(g, wsf=t(512, 4, dtype=U8)), r"block scales must be \(2, 128, 4\)"),
        # results
        ("route: wider experts", lambda g: route(g, experts=t(4, 3)), r"experts must be \(4, 2\)"),
        ("route: wider weights", lambda g: route(g, weights=t(4, 3, dtype=F32)), r"weights must be \(4, 2\)"),
        ("route: wider slots", lambda g: route(g, slots=t(4, 3)), r"slots must be \(4, 2\)"),
        ("quantize: wider codes", lambda g: quantize(g, q=t(4, 64, dtype=U8)), r"q must be \(4, 32\)"),
        ("quantize: wider codes of a fan-out", lambda g: quantize(g, fan=True, q=t(8, 64, dtype=U8)), r"q must be \(8, 32\)"),
        ("dequantize: a wider result", lambda g: dequantize(g, out=t(4, 96, dtype=BF)), r"out must be \(4, 64\)"),
        ("linear: a wider result", lambda g: linear(g, out=t(4, 16, dtype=BF)), r"out must be \(4, 8\)"),
        ("combine: a wider result", lambda g: combine(g, out=t(4, 72, dtype=BF)), r"out must be \(4, 64\)"),
        # types, counts and sizes
        ("route: rows that are not dense", lambda g: route(g, logits=t(4, 16, dtype=F32)[:, ::2]), "contiguous rows"),
        ("route: logits' type", lambda g: route(g, logits=t(4, 8, dtype=I32)), "logits must be"),
        ("route: logits' dimensions", lambda g: route(g, logits=t(8, dtype=F32)), "logits must be"),
        ("route: k of more than the experts", lambda g: route(g, k=9), "k must be"),
        ("route: k of 0", lambda g: route(g, k=0), "k must be"),
        ("route: short offsets", lambda g: route(g, offsets=t(8)), "offsets holds 32 bytes"),
        ("route: weights' type", lambda g: route(g, weights=t(4, 2)), "weights must be a tensor of"),
        ("route: short slots", lambda g: route(g, slots=t(3, 2)), "slots holds 24 bytes"),
        ("route: experts' type", lambda g: route(g, experts=t(4, 2, dtype=I64)), "experts must be a tensor of"),
        ("quantize: slots without experts", lambda g: quantize(g, slots=t(4, 2)), "come together"),
        ("quantize: experts of another shape", lambda g: quantize(g, fan=True, experts=t(4, 1)), "same shape"),
        ("quantize: slots of other tokens", lambda g: quantize(g, slots=t(5, 2), experts=t(5, 2)), "slots must be a 2-D"),
        ("quantize: slots' type", lambda g: quantize(g, fan=True, slots=t(4, 2, dtype=I64)), "slots must be a tensor of"),
        ("quantize: scales of another count", lambda g: quantize(g, scale=t(3, dtype=F32)), r"one per expert \(2\)"),
        ("quantize: scale's type", lambda g: quantize(g, scale=t(2, dtype=BF)), "scale must be a tensor of"),
        ("quantize: short codes", lambda g: quantize(g, q=t(3, 32, dtype=U8)), "q holds 96 bytes"),
        ("quantize: short block scales", lambda g: quantize(g, sf=t(128, 4, dtype=U8)), "block_scale holds 512 bytes"),
        ("quantize: activation", lambda g: quantize(g, act="relu"), "act must be"),
        ("quantize: offsets' type", lambda g: quantize(g, offsets=t(3, dtype=I64)), "offsets must be a tensor of"),
        ("quantize: offsets' dimensions", lambda g: quantize(g, offsets=t(3, 1)), "offsets must be a 1-D"),
        ("quantize: x's type", lambda g: quantize(g, x=t(4, 64, dtype=F32)), "x must be a 2-D"),
        ("quantize: an odd pair of gate and up", lambda g: quantize(g, x=t(4, 65, dtype=BF), act="silu"), "even number of columns"),
        ("dequantize: short block scales", lambda g: dequantize(g, sf=t(128, 4, dtype=U8)), "block scales holds 512 bytes"),
        ("dequantize: the result's type", lambda g: dequantize(g, out=t(4, 64)), "the output must be"),
        ("dequantize: another type than asked for", lambda g: dequantize(g, dtype=F16), "the output must be"),
        ("dequantize: a short result", lambda g: dequantize(g, out=t(3, 64, dtype=BF)), "out holds 384 bytes"),
        ("dequantize: scales of another count", lambda g: dequantize(g, scale=t(3, dtype=F32)), r"one per expert \(2\)"),
        ("linear: another count of experts", lambda g: linear(g, wq=t(3, 8, 32, dtype=U8)), "one matrix for each of 2 experts"),
        ("linear: another K", lambda g: linear(g, wq=t(2, 8, 64, dtype=U8), wsf=t(2, 128, 8, dtype=U8)), "the weight 128"),
        ("linear: the weight's type", lambda g: linear(g, wq=t(2, 8, 32, dtype=I32)), "weight_q must be a tensor of"),
        ("linear: short weight scales", lambda g: linear(g, wsf=t(1, 128, 4, dtype=U8)), "block scales holds 512 bytes"),
        ("linear: alphas of another count", lambda g: linear(g, alpha=t(5, dtype=F32)), r"one per expert \(2\)"),
        ("linear: one expert's bias", lambda g: linear(g, bias=t(8, dtype=BF)), "bias holds 16 bytes"),
        ("linear: the bias's type", lambda g: linear(g, bias=t(2, 8, dtype=F16)), "bias must be a tensor of"),
        ("linear: a short result", lambda g: linear(g, out=t(3, 8, dtype=BF)), "out holds 48 bytes"),
        ("linear: the result's type", lambda g: linear(g, out=t(4, 8)), "the output must be"),
        ("linear: short block scales", lambda g: linear(g, sf=t(128, 4, dtype=U8)), "block scales holds 512 bytes"),
        ("combine: the result's type", lambda g: combine(g, out=t(4, 64, dtype=F32)), "out must be a tensor of"),
        ("combine: fewer weights", lambda g: combine(g, weights=t(4, 1, dtype=F32)), "weights holds 16 bytes"),
        ("combine: a short addend", lambda g: combine(g, add=t(3, 64, dtype=BF)), "add holds 384 bytes"),
        ("combine: the addend's type", lambda g: combine(g, add=t(4, 64, dtype=F32)), "add must be a tensor of"),
        ("combine: rows that are not dense", lambda g: combine(g, y=t(8, 128, dtype=BF)[:, ::2]), "y must be contiguous"),
        ("combine: flat slots", lambda g: combine(g, slots=t(8)), "slots must be a 2-D"),
        ("combine: a short result", lambda g: combine(g, out=t(3, 64, dtype=BF)), "out holds 384 bytes"),
    ]


def names():
    return [c[0] for c in calls(lambda *shape, dtype=I32: None)]
