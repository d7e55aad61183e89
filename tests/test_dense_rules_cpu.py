"""Rules of the dense operators' sources that no result can show on one run."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_02_gb300", "csrc")


def source(name):
    """The file's code without comments."""
    text = open(os.path.join(CSRC, name), encoding="utf-8").read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def kernels(text):
    """(name, body) of every __global__ function."""
    out = []
    for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\((?:[^()]|\([^()]*\))*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        out.append((m.group(1), text[m.end():i]))
    return out


#: launched as programmatic dependents: what they read may be written by the launch before while they are resident
DENSE = ["dense_gemv.cu", "rmsnorm.cu", "dense_grad.cu", "dense_gemm.cuh", "dense_gemm_split.cuh", "dense_gemm_pairsplit.cuh",
         "dense_gemm_pair.cu", "activation.cuh"]


@pytest.mark.parametrize("name", DENSE)
def test_dependents_start_after_the_own_wait(name):
    """A launch lets the next one start only when its own inputs are complete: two launches overlap, never three."""
    text = source(name)
    found = kernels(text)
    assert len(found) == text.count("__global__")
    for kernel, body in found:
        assert body.count("pdl_wait()") == 1, kernel
        assert 0 <= body.index("pdl_wait()") < body.index("pdl_trigger()"), kernel


@pytest.mark.parametrize("name", DENSE)
def test_no_loads_through_the_non_coherent_path(name):
    """ld.global.nc (also as __ldg, or from a const __restrict__ pointer) needs data that nothing writes in the
    grid's lifetime, which begins before the launch ahead of it has ended."""
    text = source(name)
    for word in (".nc.", ".nc ", "__ldg", "__restrict__"):
        assert word not in text, word


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))))
def test_no_load_into_several_ctas(name):
    """Every bulk copy lands in one CTA: the library is also loaded by replica processes on several GPUs, where a copy
    with cluster multicast has no place.  (Barrier signals to both CTAs of a pair are no copies.)"""
    for m in re.finditer(r"\basm\b.*?;\s*\n", source(name), flags=re.S):
        if "cp.async.bulk" in m.group(0):
            assert "multicast" not in m.group(0)


# ------------------------------------------------------------------ sizes whose tile arithmetic would leave 32 bits
@pytest.fixture(scope="module")
def lib():
    from mixture_experts_layer_02_gb300 import build, moe
    build.build()
    return moe.load()


LAST = 2 ** 31 - 8  # the largest multiple of 8 that an int holds


@pytest.mark.parametrize("N,D,F", [(LAST, 8, 8), (2 ** 31 - 1, 8, 8), (2 ** 31 - 4095, 8, 8), (4, LAST, 8), (4, 8, LAST),
                                   (40, LAST, 8), (40, 8, LAST)])
def test_products_refuse_sizes_past_their_tile_arithmetic(lib, N, D, F):
    """Sizes rounded up to whole tiles or batches of steps have to stay below 2^31.  Placeholders for pointers: no call
    may reach a launch."""
    X, WS, big = 4096, 8192, 1 << 62
    assert lib.moe_gated_linear(X, X, X, N, D, F, 2, X, None, None, WS, big, None) == 1
    assert lib.moe_linear(X, X, None, None, N, D, F, 0, X, None, WS, big, None) == 1
    assert lib.moe_gated_linear_backward(X, X, X, X, X, X, N, D, F, 2, X, X, X, WS, big, None) == 1
    assert lib.moe_linear_backward(X, X, X, None, N, D, F, 0, X, X, None, WS, big, None) == 1
    from mixture_experts_layer_02_gb300 import moe
    for op in ("gated_linear", "linear", "gated_linear_backward", "linear_backward"):
        assert moe.workspace_size(op, N=N, D=D, Dff=F) == 0
    assert b"above 2147479552" in lib.moe_last_error_detail()


def test_products_take_sizes_up_to_there(lib):
    from mixture_experts_layer_02_gb300 import moe
    assert moe.workspace_size("linear", N=2 ** 31 - 4096, D=8, Dff=8) == 256
    assert moe.workspace_size("linear_backward", N=2 ** 31 - 4096, D=8, Dff=8) == 256 + (2 ** 31 - 4096) * 16
    assert moe.workspace_size("linear", N=4, D=2 ** 31 - 4096, Dff=8) == 256
