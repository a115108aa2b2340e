"""Kernels launched as dependents of the stream's previous kernel are alive while that one
still writes, so a load that needs memory unwritten for a kernel's life (``__ldg``) may
take only what no kernel of a serving step writes: tables of cosines, head scales, masks.
An append also turns queries in place, which rules it out for them on their own."""

import pathlib
import re

import pytest

import decode_attention_flash_gb300 as da

CSRC = pathlib.Path(da.__file__).parent / "csrc"
DEPENDENT = sorted(f.name for f in CSRC.glob("*.cu") if "wait_for_previous_kernel()" in f.read_text())
CONSTANT = re.compile(r"(row|row2|p\.cos_sin|p\.[kv]_scale|p\.mask_window|p\.mask_sink|p\.alibi_slopes)\b")


def loads(text):
    """The arguments of the read-only loads of a source without its comments."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__ldg\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        yield text[m.end():at - 1]


def test_there_are_dependent_kernels():
    assert DEPENDENT == ["cache_rows.cu", "fp4_split.cu", "tables.cu"]


@pytest.mark.parametrize("name", DEPENDENT)
def test_read_only_loads_take_constants(name):
    text = (CSRC / name).read_text()
    assert [a for a in loads(text) if not CONSTANT.match(a)] == []
    assert "__restrict__" not in text and "global.nc" not in text
