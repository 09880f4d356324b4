"""CPU checks of the expert operators' binding: each refusal with its words, so
that a call refused for another reason does not pass for it."""
import pytest
import torch

from experts_refusals import calls, names


@pytest.fixture(scope="module")
def gnq():
    from nvfp4_quant_gemma_gb300 import build
    build.build()
    import nvfp4_quant_gemma_gb300 as pkg
    return pkg


@pytest.mark.parametrize("i", range(len(names())), ids=names())
def test_the_binding_refuses_in_these_words(gnq, i):
    _, call, words = calls(lambda *shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype))[i]
    with pytest.raises(ValueError, match=words):
        call(gnq)
