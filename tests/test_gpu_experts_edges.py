"""GPU tests of the expert operators where they could go wrong unseen: refusals
of device tensors, shapes that the kernels index, offsets in no order, sums that
must not depend on the batch."""
import pytest
import torch

import oracle
from experts_ref import scale_rows
from experts_refusals import calls, names
from gnq_testutil import u8
from test_gpu_experts import ALL, _operands, fp32, ints
from test_gpu_operators import SENT, Guarded

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
    pkg.read_device_error()
    return pkg


# ---------------------------------------------------------------------------
# shapes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("i", range(len(names())), ids=names())
def test_the_binding_refuses_device_tensors_in_these_words(gnq, i):
    """The one-expression check of a call's arguments lets none of them by."""
    _, call, words = calls(lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype, device="cuda"))[i]
    with pytest.raises(ValueError, match=words):
        call(gnq)


def test_shapes_that_hold_the_call_s_matrices(gnq):
    """More rows, flat buffers of the very size and leading dimensions give the
    bits of the plain shapes."""
    M, k, H, E = 6, 2, 64, 3
    y, slots = torch.randn(M * k, H, device="cuda"), torch.randperm(M * k, device="cuda").reshape(M, k).int()
    w, add = torch.rand(M + 3, k, device="cuda"), torch.randn(M + 2, H, device="cuda")
    want = gnq.expert_combine(y, slots, w[:M].clone(), add=add[:M].clone())
    for weights, a in ((w, add), (w[:M].reshape(-1).clone(), add[:M].reshape(-1).clone()),
                       (w[:M].clone().view(2, 3, k), add[:M].clone().view(2, 3, H))):
        assert torch.equal(gnq.expert_combine(y, slots, weights, add=a), want)
    out = torch.zeros(2, 3, H, device="cuda")
    assert torch.equal(gnq.expert_combine(y, slots, w, add=add, out=out).view(M, H), want)
    out = torch.zeros(M * H + 5, device="cuda")
    assert torch.equal(gnq.expert_combine(y, slots, w, add=add, out=out)[:M * H].view(M, H), want)

    offsets, q, sf, wq, wsf = _operands([3, 0, 4], 200, 128, 1)
    args, o = [v.cuda() for v in (q, sf, wq)], ints(offsets)
    bias = torch.randn(E, 200, device="cuda").to(torch.bfloat16)
    want = gnq.nvfp4_expert_linear(*args, wsf.cuda(), fp32([0.01]), o, bias=bias)
    more = torch.cat((wsf.view(torch.uint8), torch.zeros(1, 256, 8, dtype=torch.uint8))).cuda()
    for scales, b in ((wsf.cuda().reshape(-1), bias.reshape(-1)), (wsf.cuda().reshape(E * 256, 8), torch.cat((bias, bias))),
                      (more, bias)):
        assert torch.equal(gnq.nvfp4_expert_linear(*args, scales, fp32([0.01]), o, bias=b), want)


# ---------------------------------------------------------------------------
# offsets in no order
# ---------------------------------------------------------------------------
def _ascending(E, R):
    return [R * e // E for e in range(E + 1)]


def _with(offsets, **at):
    offsets = list(offsets)
    for i, v in at.items():
        offsets[int(i[1:])] = v
    return offsets


BAD = {
    "falling": [0, 5, 3, 9], "negative": [0, -4, 4, 9], "far": [0, 3, 6, 1 << 30], "behind the rows": [0, 3, 6, 10],
    "a late start": [2, 3, 6, 9], "an early start": [-5, 3, 6, 9], "far and back": [0, 1 << 30, -(1 << 30), 9],
    "falling among many": _with(_ascending(1024, 9), i1000=3), "behind the rows among many": _with(_ascending(700, 9), i700=10),
    "a late start among many": _with(_ascending(300, 9), i0=1),
}


@pytest.mark.parametrize("bad", BAD.values(), ids=BAD.keys())
def test_offsets_in_no_order_are_reported_by_each_operator(gnq, bad):
    """Each call sets the word by itself; rows in nobody's bounds stay as they were."""
    E, R, H = len(bad) - 1, 9, 128
    o, s = ints(bad), fp32([9.0])
    x = torch.randn(R, H, device="cuda").to(torch.bfloat16)
    held = {r for e in range(E) for r in range(max(bad[e], 0), min(bad[e + 1], R))}
    slots = torch.arange(R, device="cuda").reshape(R, 1).int()
    owner = [next((e for e in range(E) if max(bad[e], 0) <= r < bad[e + 1]), -1) for r in range(R)]
    q0 = torch.zeros(R, H // 2, dtype=torch.uint8, device="cuda")
    sf0 = torch.zeros(scale_rows(R, E), H // 16, dtype=torch.uint8, device="cuda")
    gnq.read_device_error()
    for call in (lambda q, sf, back: gnq.expert_quantize(x, o, s, out=(q, sf)),
                 lambda q, sf, back: gnq.expert_quantize(torch.cat((x, x), 1), o, s, act="silu", out=(q, sf)),
                 lambda q, sf, back: gnq.expert_quantize(x, o, s, out=(q, sf), slots=torch.where(ints(owner)[:, None] < 0, -1, slots),
                                                         experts=ints(owner)[:, None]),
                 lambda q, sf, back: gnq.expert_dequantize(q0, sf0, o, s, out=back),
                 lambda q, sf, back: gnq.expert_dequantize(q0, sf0, o, s, out=back.view(torch.uint8)[:, :H].contiguous()
                                                           .view(torch.float8_e4m3fn))):
        G = Guarded()
        q, sf, back = G((R, H // 2), torch.uint8), G((scale_rows(R, E), H // 16), torch.uint8), G((R, H), torch.bfloat16)
        call(q, sf, back)
        torch.cuda.synchronize()
        G.check()
        assert gnq.read_device_error() == 2
        for buf in (q, back):
            for r in range(R):
                assert r in held or (u8(buf)[r] == SENT).all()


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("bad", BAD.values(), ids=BAD.keys())
def test_the_product_of_offsets_in_no_order_writes_nothing(gnq, bad, kernel):
    E, R, N, K = len(bad) - 1, 9, 136, 128
    q = torch.zeros(R, K // 2, dtype=torch.uint8, device="cuda")
    sf = torch.zeros(scale_rows(R, E), K // 16, dtype=torch.uint8, device="cuda")
    wq = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    wsf = torch.zeros(E, 256, K // 16, dtype=torch.uint8, device="cuda")
    G = Guarded()
    y = G((R, N), torch.bfloat16)
    gnq.read_device_error()
    gnq.set_linear_policy(kernel)
    try:
        gnq.nvfp4_expert_linear(q, sf, wq, wsf, fp32([1.0]), ints(bad), out=y)
        torch.cuda.synchronize()
    finally:
        gnq.set_linear_policy(0)
    G.check()
    assert gnq.read_device_error() == 2 and (u8(y) == SENT).all()


@pytest.mark.parametrize("E", [3, 300, 700, 1024])
def test_offsets_in_order_are_not_reported(gnq, E):
    """Bounds of all kinds that are right: empty experts, rows of nobody."""
    R, H = 9, 128
    x = torch.randn(R, H, device="cuda").to(torch.bfloat16)
    for offsets in (_ascending(E, R), [0] * E + [R], [0] + [R] * E, [0] * (E + 1), _ascending(E, 4)):
        o, s = ints(offsets), fp32([9.0])
        q, sf = gnq.expert_quantize(x, o, s)
        gnq.expert_dequantize(q, sf, o, s)
        owner = torch.searchsorted(torch.tensor(offsets[1:]), torch.arange(R), right=True)
        owner = torch.where(owner < E, owner, -1).int().cuda()[:, None]
        slots = torch.where(owner >= 0, torch.arange(R, device="cuda").int()[:, None], -1)
        gnq.expert_quantize(x, o, s, slots=slots, experts=owner)
        torch.cuda.synchronize()
        assert gnq.read_device_error() == 0


# ---------------------------------------------------------------------------
# the combination of large batches
# ---------------------------------------------------------------------------
LARGE = (2500, 520)  # tokens and columns: more units than the instance of small batches takes


def _combination(M, H, k, Y, seed):
    g = torch.Generator().manual_seed(seed)
    y = torch.randn(M * k, H, generator=g).to(ALL[Y])
    slots = torch.randperm(M * k, generator=g).reshape(M, k)
    slots[::7, k // 2] = -1
    slots[5] = -1
    return y, slots, torch.rand(M, k, generator=g)


@pytest.mark.parametrize("k", [1, 2, 3, 8, 9, 32])
@pytest.mark.parametrize("Y,O", [("bf16", "bf16"), ("fp32", "fp32")])
def test_a_token_s_combination_does_not_depend_on_the_batch(gnq, k, Y, O):
    M, H = LARGE
    y, slots, w = _combination(M, H, k, Y, k)
    add = torch.randn(M, H).to(ALL[O]).cuda()
    y, slots, w = y.cuda(), slots.int().cuda(), w.cuda()
    whole = gnq.expert_combine(y, slots, w, add=add)
    for a, z in ((0, 1), (0, 40), (M - 200, M)):
        part = gnq.expert_combine(y, slots[a:z].contiguous(), w[a:z].contiguous(), add=add[a:z].contiguous())
        assert torch.equal(part, whole[a:z])
