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
