"""Rules of the kernels' sources whose breach is a race, which no run has to show (host side, no GPU)."""
from __future__ import annotations

import glob
import os
import re

import pytest

from wna16_grouped_gemm_gb300 import build

SOURCES = sorted(glob.glob(os.path.join(build.CSRC, "*.cu")))


def code_of(path):
    """The source without comments and strings' contents."""
    with open(path) as f:
        s = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", lambda m: "\n" * m.group().count("\n"), s, flags=re.S)


def bodies(s):
    """(name, body) of every __global__ function that is defined in s."""
    for m in re.finditer(r"__global__\b", s):
        name = re.search(r"\b(\w+_kernel)\s*\(", s[m.end():m.end() + 600])
        at = s.find("{", m.end())
        semicolon = s.find(";", m.end())
        if at < 0 or (0 <= semicolon < at):
            continue
        depth, i = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(s[i], 0)
            i += 1
            if depth == 0:
                break
        yield name.group(1) if name else "?", s[at:i]


def test_kernels_are_found():
    assert sum(len(list(bodies(code_of(p)))) for p in SOURCES) >= 25


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_a_cluster_has_started_before_its_shared_memory_is_reached(path):
    """A block of a cluster may reach another's shared memory once a barrier of the cluster shows that it has
    started: cluster_sync(), or cluster_wait() behind a cluster_arrive()."""
    for name, body in bodies(code_of(path)):
        first = body.find("map_shared(")
        if first < 0:
            continue
        before = body[:first]
        split = before.find("cluster_arrive()")
        assert "cluster_sync()" in before or 0 <= split < before.find("cluster_wait()"), name


def signature_of(s, name):
    at = s.index("(", s.index(name + "("))
    return s[at:s.index("{", at)]


@pytest.mark.parametrize("path", SOURCES + sorted(glob.glob(os.path.join(build.CSRC, "*.cuh"))), ids=os.path.basename)
def test_inputs_are_loaded_coherently(path):
    """A kernel that starts before the one ahead of it ends (pdl_wait) reads what that one writes: such data changes
    during the kernel's life, which the non-coherent path does not allow (__ldg, .nc, or a compiler's choice of them for a const
    __restrict__ argument), and a compiler may move its loads ahead of the wait."""
    code = code_of(path)
    kernels = [name for name, body in bodies(code) if "pdl_wait()" in body]
    if kernels or path.endswith(".cuh"):
        assert "__ldg" not in code and ".nc." not in code
    for name in kernels:
        assert not re.search(r"const[\w\s:]*\*\s*__restrict__", signature_of(code, name)), name


@pytest.mark.parametrize("name,least", [("sort_tokens.cu", 6), ("linear_f8.cuh", 3), ("linear_f8_thin.cu", 1), ("linear_f8_wide.cu", 1),
                                        ("gemm.cu", 10), ("kernels.cu", 6)])
def test_indices_from_device_data_are_checked_in_the_bounds_checked_build(name, least):
    code = code_of(os.path.join(build.CSRC, name))
    assert len(re.findall(r"\b(?:row_)?in_bounds\(", code)) >= least


def test_only_the_bounds_checked_build_has_the_checks_word():
    from wna16_grouped_gemm_gb300 import binding
    build.build()
    build.build(debug=True)
    assert hasattr(binding.load_debug_library(), "wna16_moe_debug_index_status")
    assert not hasattr(binding.load_library(), "wna16_moe_debug_index_status")
