"""GPU tests of the expert operators where they could go wrong unseen: refusals
of device tensors, shapes that the kernels index, offsets in no order, sums that
must not depend on the batch, and the instances that only large batches, other
types, other alignments or combined options reach."""
import pytest
import torch

import oracle
from experts_ref import scale_rows
from experts_refusals import calls, names
from gnq_testutil import DTYPES, u8
from operators_ref import assert_within, rounding
from test_gpu_experts import (ALL, COUNTS, _check_packed, _fan, _logits, _operands, _run_linear, _values, fp32, ints,
                              offsets_of, random_rows, route64)
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


@pytest.mark.parametrize("Y,O", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16"), ("fp32", "fp16")])
@pytest.mark.parametrize("add", ["none", "apart", "in place"])
@pytest.mark.parametrize("k", [5, 8])
def test_combine_large_batches(gnq, k, add, Y, O):
    M, H = LARGE
    y, slots, w = _combination(M, H, k, Y, 11 + k)
    a = torch.randn(M, H, generator=torch.Generator().manual_seed(k)).to(ALL[O])
    G = Guarded()
    out = G((M, H), ALL[O])
    if add == "in place":
        out.copy_(a)
    gnq.expert_combine(y.cuda(), slots.int().cuda(), w.cuda(), out=out, add={"none": None, "apart": a.cuda(), "in place": out}[add])
    torch.cuda.synchronize()
    G.check()
    assert gnq.read_device_error() == 0
    rows = y.double()[slots.clamp(min=0)] * (w.double() * (slots >= 0))[..., None]
    want, mag = rows.sum(1), rows.abs().sum(1)
    if add != "none":
        want, mag = want + a.double(), mag + a.double().abs()
    # a term is rounded in its product, in its pair, in the sum of the pairs and with `add`: at most k + 1 times
    err = (k + 2) * 2.0 ** -24 * mag
    assert_within(out, want, err + rounding(want.abs() + err, ALL[O]), "out")


# ---------------------------------------------------------------------------
# the router
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,E,k", [(50001, 24, 8), (40000, 300, 8), (20003, 128, 32)])
def test_route_places_long_chunks(gnq, M, E, k, dtype):
    """More choices a warp than it keeps in registers: places wait in the slots."""
    v = _logits(M, E, dtype, M, ties=True)
    v[::11] = -float("inf")
    v[3::13, 2:] = -float("inf")
    G = Guarded()
    out = (G((M, k), torch.int32), G((M, k), torch.float32), G((E + 1,), torch.int32), G((M, k), torch.int32))
    gnq.expert_route(v.cuda(), k, out=out)
    torch.cuda.synchronize()
    G.check()
    top = torch.sort(v.double() + 0.0, dim=1, descending=True, stable=True)
    experts = torch.where(top.values[:, :k] == -float("inf"), -1, top.indices[:, :k]).int()
    flat = experts.reshape(-1)
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    used = int((flat >= 0).sum())
    slots = torch.full((M * k,), -1, dtype=torch.int32)
    slots[order[:used]] = torch.arange(used, dtype=torch.int32)
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64), torch.bincount(flat[flat >= 0].long(), minlength=E).cumsum(0)))
    assert torch.equal(out[0].cpu(), experts) and torch.equal(out[2].cpu(), offsets.int())
    assert torch.equal(out[3].cpu(), slots.reshape(M, k))


@pytest.mark.parametrize("M", [20, 1300])
@pytest.mark.parametrize("E", [40, 256, 1000])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_route_nan_and_infinities_of_every_type(gnq, dtype, renormalize, E, M):
    """NaN of either sign above +inf, its index deciding among equals; a token
    that has one, or +inf, gets NaN weights, and no other token does."""
    k, T = 4, ALL[dtype]
    v = _logits(M, E, dtype, E)
    clean = gnq.expert_route(v.cuda(), k, renormalize=renormalize)
    nan = {"bf16": (0x7FC0, -0x3F), "fp16": (0x7E01, -0x1FF), "fp32": (0x7FC00001, -0x3FFFFF)}[dtype]
    bits = v.view(torch.int32 if dtype == "fp32" else torch.int16)
    bits[3, 9] = nan[0]
    bits[4, 38] = nan[1]                      # negative
    bits[8, 30], bits[8, 31] = nan[1], nan[0]
    v[5, 2] = float("inf")
    v[6, 1], v[6, 2], v[6, 3] = float("inf"), float("inf"), -float("inf")
    v[7, 20] = float("inf")
    bits[7, 39] = nan[1]
    v[11] = -float("inf")
    bits[11, 6] = nan[0]
    v[12] = -float("inf")
    v[12, 17] = torch.finfo(T).min
    odd = torch.zeros(M, dtype=torch.bool)
    odd[[3, 4, 5, 6, 7, 8, 11]] = True
    assert torch.isnan(v).any(1).sum() == 5
    experts, weights, offsets, slots = (t.cpu() for t in gnq.expert_route(v.cuda(), k, renormalize=renormalize))
    e64, _, o64, s64 = route64(v, k, renormalize, 1.0)
    assert torch.equal(experts, e64) and torch.equal(offsets, o64) and torch.equal(slots, s64)
    assert torch.equal(torch.isnan(weights), odd[:, None] & (experts >= 0))
    assert weights[11, 1:].tolist() == [0.0] * 3 and weights[12].tolist() == [1.0, 0.0, 0.0, 0.0]
    keep = ~odd
    keep[12] = False
    assert torch.equal(weights[keep], clean[1].cpu()[keep])


# ---------------------------------------------------------------------------
# the way back
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T", [torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn])
@pytest.mark.parametrize("counts,K", [("tiles", 320), ("few", 64), ("many", 64)])
def test_dequantize_to_16_byte_alignment(gnq, counts, K, T):
    """A result that is 16-byte but not 32-byte aligned has the same bits."""
    offsets = offsets_of(COUNTS[counts])
    R = offsets[-1] + 2
    q, sf = (v.cuda() for v in random_rows(offsets, R, K, 3))
    G = Guarded()
    outs = G((R, K), T), G((R, K), T, shift=16)
    assert outs[0].data_ptr() % 32 == 0 and outs[1].data_ptr() % 32 == 16
    for out in outs:
        gnq.expert_dequantize(q, sf, ints(offsets), fp32([3.0]), out=out)
    torch.cuda.synchronize()
    G.check()
    assert (u8(outs[0]) == u8(outs[1])).all()


# ---------------------------------------------------------------------------
# quantization and products
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("counts,H,k", [("few", 64, 3), ("tiles", 192, 8), ("single", 2048, 5), ("many", 64, 32)])
def test_quantize_activated_and_fanned_out(gnq, counts, H, k, act, dtype):
    """The gated activation of a token, with the scale of each of its experts."""
    offsets, slots, experts = _fan(COUNTS[counts], k, 2)
    E, (M, k) = len(offsets) - 1, slots.shape
    x = _values(M, 2 * H, DTYPES[dtype], M).cuda()
    for shared in (False, True):
        scales = [168.0] * E if shared else [50.0 + 13.0 * (e % 9) for e in range(E)]
        G = Guarded()
        out = G((M * k, H // 2), torch.uint8), G((scale_rows(M * k, E), H // 16), torch.float8_e4m3fn)
        q, bs = gnq.expert_quantize(x, ints(offsets), fp32(scales[:1] if shared else scales), slots=slots.int().cuda(),
                                    experts=experts.int().cuda(), act=act, out=out)
        v = gnq.gated_act_quant(x, None, "none", act=act)[2].cpu()
        torch.cuda.synchronize()
        G.check()
        y = torch.zeros(offsets[-1], H, dtype=v.dtype)
        t, j = (slots >= 0).nonzero(as_tuple=True)
        y[slots[t, j]] = v[t]
        _check_packed(q, bs, y, scales, offsets, dtype)
    assert gnq.read_device_error() == 0


@pytest.mark.parametrize("N", [1, 8, 24, 40, 248, 264])
@pytest.mark.parametrize("T", [torch.bfloat16, torch.float16, torch.float32])
def test_pairs_of_few_columns(gnq, T, N):
    """The pair kernel where its tile of 256 columns is clipped, in tile stores
    (16-bit rows that are a multiple of 16 bytes) and without."""
    gnq.set_linear_policy(2)
    try:
        for counts in ([1], [33, 0, 300], [31, 64, 449]):
            _run_linear(gnq, counts, N, 320, T, seed=N)
    finally:
        gnq.set_linear_policy(0)
