"""Shared-memory arrays that are read or written in 16-byte units say so where they are
declared: an array of floats has the place the others before it leave, which may be any
multiple of 4, and a 16-byte access elsewhere is a fault (CPU: reads the sources)."""
import glob
import os
import re

import pytest

from speculative_decode_verify_sdv_gb300 import build

SOURCES = sorted(glob.glob(os.path.join(build.CSRC, "*.cu")) + glob.glob(os.path.join(build.CSRC, "*.cuh")))
WIDE = r"(?:float4|uint4|int4|double2|ulonglong2)"


def plain_arrays(text):
    """Names of shared arrays without an alignment and with elements of less than 16 bytes."""
    names = set()
    for m in re.finditer(r"__shared__\s+([^;]*);", text):
        decl = m.group(1)
        if "alignas" in decl or re.match(rf"(?:volatile\s+)?{WIDE}\b", decl):
            continue
        names |= set(re.findall(r"(\w+)\s*\[", decl.split("=")[0]))
    return names


def wide_accesses(text):
    """Arrays whose elements are accessed as 16-byte units: a cast of &name[...] or of name."""
    return set(re.findall(rf"reinterpret_cast<(?:const\s+)?{WIDE}\s*\*>\(\s*&?\s*(\w+)\b", text))


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(p) for p in SOURCES])
def test_arrays_accessed_in_16_byte_units_are_aligned(path):
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert not plain_arrays(text) & wide_accesses(text)


def test_a_plain_array_is_found():
    text = "__shared__ alignas(16) float a[4], b[8]; __shared__ float c[3 * 4]; x = *reinterpret_cast<const float4*>(\n &c[4]);"
    assert plain_arrays(text) & wide_accesses(text) == {"c"}
