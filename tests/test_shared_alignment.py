"""Shared arrays that kernels read by wider types than their own declare the alignment for it."""
import glob
import os
import re

import pytest

import gated_causal_softmax_gb300

CSRC = os.path.join(os.path.dirname(gated_causal_softmax_gb300.__file__), "csrc")
WIDTH = {"uint2": 8, "int2": 8, "float2": 8, "uint4": 16, "int4": 16, "float4": 16}


@pytest.mark.parametrize("name", sorted(map(os.path.basename, glob.glob(os.path.join(CSRC, "*.cu*")))))
def test_shared_arrays_read_by_wider_types(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    arrays = {}
    for decl in re.finditer(r"__shared__\s+(?:__align__\((\d+)\)\s*)?([\w:]+)\s+([^;{]+);", text):
        for array in re.findall(r"(\w+)\[", decl.group(3)):
            arrays[array] = int(decl.group(1) or WIDTH.get(decl.group(2), 0))
    for wide, array in re.findall(r"reinterpret_cast<(?:const )?(\w+)\s*\*>\(&?(\w+)\b(?!\.)", text):
        if wide in WIDTH and array in arrays:
            assert arrays[array] >= WIDTH[wide], (array, wide)
