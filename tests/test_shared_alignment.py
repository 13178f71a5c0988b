"""CPU check of the kernels' sources: a shared array of 8- or 16-bit elements
has their alignment alone, so it is read and written through wider pointers
only where its declaration asks for more."""
import re

import pytest

from extreme_label_sparse_gb300 import _build

DECL = re.compile(r"(?<!extern )__shared__\s+(alignas\(\d+\)\s+|__align__\(\d+\)\s+)?"
                  r"(?:unsigned char|char|u?int8_t|u?int16_t|__half|__nv_bfloat16)\s+(\w+)\s*\[")


@pytest.mark.parametrize("source", sorted(p.name for p in _build.CSRC.glob("*.cu*")))
def test_narrow_shared_arrays_are_not_accessed_by_wider_words(source):
    text = (_build.CSRC / source).read_text()
    for aligned, name in DECL.findall(text):
        wide = re.findall(r"reinterpret_cast<(?:const )?(?:u?int32_t|u?int64_t|float\d?|u?int\d) \*>\(\s*&?" + name + r"\b", text)
        assert aligned or not wide, (source, name, wide)
