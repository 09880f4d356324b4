"""CPU checks of the operators around the NVFP4 linear: what their entry points
refuse beyond single arguments, and host code that a GPU test cannot make fail."""
import ctypes
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, i64, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from nvfp4_quant_gemma_gb300 import build
    build.build()
    import nvfp4_quant_gemma_gb300 as pkg
    return pkg.load()


def test_split_timeout_hook_takes_a_cta_or_off(lib):
    f = lib.gnq_inject_split_timeout
    assert f(8) == 2 and f(-2) == 2
    assert f(7) == 0 and f(-1) == 0


# Pointers that are never dereferenced: every call below is refused.  M = 4,
# H = K = N = 64: x and the 16-bit outputs hold 512 bytes, FP8 codes 256,
# NVFP4 codes 128, block scales 512 (padding rows included).
A, B, C, D, E = (0x100000 * i for i in range(1, 6))


def sandwich(lib, **kw):
    a = dict(x=A, r=B, ro=None, wp=None, w=C, gate=None, gs=0, scale=C + 0x1000, mode=0, wy=0, q=D, bs=None, y=None)
    a.update(kw)
    return lib.gemma_sandwich_norm_quant(P(a["x"]), P(a["r"]), P(a["ro"]), P(a["wp"]), P(a["w"]), P(a["gate"]),
                                         i64(a["gs"]), F(1.0), F(1e-6), P(a["scale"]), a["mode"], a["wy"], P(a["q"]),
                                         P(a["bs"]), P(a["y"]), i64(4), i64(64), 0, None)


@pytest.mark.parametrize("kw", [
    dict(q=A), dict(q=B), dict(ro=E, q=E), dict(ro=E, q=B), dict(q=C), dict(q=C + 0x1000),  # codes over x, residual(s), w, scale
    dict(q=A + 256), dict(q=A - 240), dict(q=B + 496),                           # in part
    dict(ro=B + 16), dict(ro=A - 496), dict(ro=C - 16), dict(wp=E, ro=E),        # the new residual
    dict(wy=1, y=D), dict(wy=1, y=B + 256), dict(wy=1, ro=E, y=E + 16), dict(ro=E, wy=1, y=B),  # y
    dict(mode=1, bs=D + 64), dict(mode=1, bs=A + 508), dict(mode=2, bs=D + 252),  # block scales
    dict(gate=B + 480), dict(gate=E, gs=64, q=E + 256), dict(gate=E, gs=128, q=E + 0x240, ro=B),  # gate rows
    dict(gate=E, gs=128, mode=1, q=E + 0x110, bs=A + 0x4000),                    # q crosses into the gate's next row
])
def test_sandwich_refuses_outputs_over_what_it_uses(lib, kw):
    assert sandwich(lib, **kw) == 5


@pytest.mark.parametrize("kw", [
    dict(q=A), dict(q=A + 0x80), dict(q=A - 0xF0), dict(q=B), dict(mode=1, bs=C), dict(mode=1, bs=A + 0x100),
    dict(stride=512, q=A + 0x400), dict(stride=512, q=A + 0x380), dict(stride=512, q=A + 0xC00),  # rows far apart
    dict(stride=512, q=A + 0x340),                                                        # ends in the next row
])
@pytest.mark.parametrize("act", [0, 1])
def test_quantize_and_gated_refuse_outputs_over_what_they_use(lib, kw, act):
    a = dict(x=A, stride=128, scale=B, mode=0, q=C, bs=D)
    a.update(kw)
    if act:
        st = lib.gated_act_quant(P(a["x"]), i64(a["stride"]), act, P(a["scale"]), a["mode"], 0, P(a["q"]), P(a["bs"]),
                                 None, i64(4), i64(64), 0, None)
    else:
        st = lib.gnq_quantize(P(a["x"]), i64(a["stride"]), P(a["scale"]), a["mode"], P(a["q"]), P(a["bs"]), i64(4),
                              i64(64), 0, None)
    assert st == 5


@pytest.mark.parametrize("kw", [dict(wy=1, y=A + 16), dict(wy=1, y=C), dict(wy=1, y=B - 496), dict(mode=-1, y=A + 128)])
def test_gated_refuses_y_over_what_it_uses(lib, kw):
    a = dict(mode=0, wy=0, y=None)
    a.update(kw)
    assert lib.gated_act_quant(P(A), i64(128), 1, P(B), a["mode"], a["wy"], P(C), P(D), P(a["y"]), i64(4), i64(64), 0,
                               None) == 5


@pytest.mark.parametrize("out", [A, A + 112, A - 496, B + 496, C])
def test_dequantize_refuses_an_output_over_what_it_reads(lib, out):
    assert lib.gnq_nvfp4_dequantize(P(A), P(B), P(C), P(out), i64(4), i64(64), 0, None) == 5


@pytest.mark.parametrize("y", [A, A + 112, B + 496, C + 2032, D - 496, E, E + 0x1000 - 496])
def test_linear_refuses_an_output_over_what_it_reads(lib, y):
    assert lib.nvfp4_linear(P(A), P(B), P(C), P(D), P(E), P(E + 0x1000), P(y), i64(4), i64(64), i64(64), 0, 0, None) == 5


def test_a_failed_question_to_the_runtime_is_asked_again(tmp_path):
    """Resident clusters (and with them the split of a product) are asked for
    once per device; one failed answer must not stay for the process."""
    exe = tmp_path / "host_helpers"
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-x", "c++", os.path.join(ROOT, "tests", "c", "host_helpers.cpp"), "-I",
                    os.path.join(ROOT, "nvfp4_quant_gemma_gb300", "csrc"), "-I", os.path.join(cuda, "include"), "-o",
                    str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and "host helpers ok" in res.stdout, res.stderr
    linear = open(os.path.join(ROOT, "nvfp4_quant_gemma_gb300", "csrc", "gnq_linear.cu")).read()
    body = linear[linear.index("int resident_clusters("):]
    assert "answer_once(" in body[:body.index("\n}")]


def test_no_cta_reads_the_shared_memory_of_a_peer():
    """A read of another CTA's shared memory has to be over before that CTA
    leaves, and a relaxed arrival on the cluster barrier does not say so: CTAs
    store into their peers instead, and the next arrival releases it.  Read off
    the sources, as a GPU could only show a slip by faulting."""
    csrc = os.path.join(ROOT, "nvfp4_quant_gemma_gb300", "csrc")
    stores = 0
    for name in sorted(os.listdir(csrc)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(csrc, name)).read())
        assert "ld.shared::cluster" not in text, name
        for store in re.finditer(r"(?<!void )\bst_cluster_\w+\(", text):
            arrival = re.search(r"\bcluster_arrive_(\w+)\(", text[store.end():])
            assert arrival and arrival.group(1) == "release", name
            stores += 1
    assert stores >= 3  # a row's sums, and the parts and the status of a split product


def test_linear_policy_and_query_arguments(lib):
    f = lib.gnq_set_linear_policy
    assert f(3) == 2 and f(-1) == 2
    assert f(2) == 0 and f(0) == 0
    out = [ctypes.byref(ctypes.c_int()) for _ in range(3)]
    q = lambda M=16, N=64, K=64, t=0, o=out: lib.gnq_query_linear(i64(M), i64(N), i64(K), t, *o)
    assert q(o=(None, *out[1:])) == 1 and q(t=3) == 3 and q(t=-1) == 3
    assert q(M=0) == 2 and q(N=0) == 2 and q(K=96) == 2 and q(K=65600) == 2
    assert q() in (0, 7)  # a choice, or no device here
