"""GPU tests of the expert operators where they could go wrong unseen: refusals
of device tensors and shapes that the kernels index."""
import pytest
import torch

import oracle
from experts_refusals import calls, names
from test_gpu_experts import _operands, fp32, ints

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
