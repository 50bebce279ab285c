"""Arrays in shared memory that are read as vectors are declared with a vector's alignment: an array of 4-byte elements
lies at any multiple of 4, and where a compiler puts it is not for the code to rely on. CPU only, from the sources."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "io_aware_exact_13_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))
SIZE = {"uint8_t": 1, "int": 4, "uint32_t": 4, "float": 4, "uint64_t": 8, "int2": 8, "uint2": 8, "float2": 8}
VECTORS = {"int2": 8, "uint2": 8, "float2": 8, "int4": 16, "uint4": 16, "float4": 16}


def unaligned(text):
    """Names of shared arrays that are cast to a vector wider than their declared alignment."""
    bad = []
    declared = re.findall(r"__shared__\s+(?:__align__\((\d+)\)\s+)?(\w+)\s+([^;]*);", text)
    for align, kind, names in declared:
        have = int(align) if align else SIZE.get(kind, 16)
        for name in re.findall(r"(\w+)\s*(?:\[[^\]]*\])+", names):
            for vector in re.findall(r"reinterpret_cast<(?:const\s+)?(\w+)\s*\*>\(\s*&?" + name + r"\b", text):
                if VECTORS.get(vector, 0) > have:
                    bad.append((name, vector))
    return bad


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_shared_arrays_read_as_vectors_are_aligned(path):
    with open(path) as f:
        assert unaligned(f.read()) == []


def test_a_planted_cast_is_found():
    text = "__shared__ int a[8]; __shared__ __align__(16) int b[8]; reinterpret_cast<const int4 *>(a)[0]; reinterpret_cast<int4 *>(b)[1];"
    assert unaligned(text) == [("a", "int4")]
