"""Shared arrays of the kernels that are read through a wider type have its alignment
declared, rather than by the place that the compiler happens to give them."""
import glob
import os
import re

from gqa_attention_kv_split_gb300 import build_lib

BYTES = {"float": 4, "int": 4, "uint32_t": 4, "int32_t": 4, "uint16_t": 2, "uint8_t": 1, "uint64_t": 8, "int64_t": 8}
WIDE = {"float2": 8, "uint2": 8, "int2": 8, "float4": 16, "uint4": 16, "int4": 16}


def test_arrays_read_through_a_wider_type_are_aligned():
    bad = []
    for path in glob.glob(os.path.join(build_lib.CSRC, "*.cu*")):
        src = re.sub(r"//.*", "", open(path).read())
        for align, scalar, name in re.findall(r"__shared__\s+(?:(?:alignas|__align__)\((\d+)\)\s+)?(\w+)\s+(\w+)\s*\[", src):
            have = int(align or BYTES.get(scalar, 16))
            for wide in re.findall(r"reinterpret_cast<(?:const\s+)?(\w+)\s*\*>\(&?" + name + r"\b", src):
                if WIDE.get(wide, 0) > have:
                    bad.append((os.path.basename(path), name, wide))
    assert not bad
