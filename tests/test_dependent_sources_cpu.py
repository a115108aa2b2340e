"""Every source whose kernels are launched as dependents of the stream's previous kernel, its headers too:
each kernel waits before it does anything else, and read-only loads take constants alone (what no kernel of a serving
step writes: tables of cosines, head scales, masks)."""

import ctypes
import pathlib
import re

import pytest

import decode_attention_flash_gb300 as da
from test_dependent_loads_cpu import CONSTANT, loads

CSRC = pathlib.Path(da.__file__).parent / "csrc"
SOURCES = ["block8_split.cu", "cache_blocks.cu", "cache_rows.cu", "cache_rows.cuh", "fp4_split.cu", "stream_split.cuh",
           "tables.cu", "verify.cu"]


def test_dependent_launches_are_in_these_sources():
    launch = re.compile(r"launch_dependent\(|ProgrammaticStreamSerialization;|ProgrammaticStreamSerialization\b")
    found = sorted(f.name for f in CSRC.glob("*.cu") if launch.search(f.read_text()))
    assert found == [s for s in SOURCES if s.endswith(".cu")]


@pytest.mark.parametrize("name", SOURCES)
def test_read_only_loads_take_constants(name):
    text = (CSRC / name).read_text()
    assert [a for a in loads(text) if not CONSTANT.match(a)] == []
    assert "__restrict__" not in text and "global.nc" not in text


@pytest.mark.parametrize("name", [s for s in SOURCES if s.endswith(".cu")])
def test_kernels_wait_before_they_load(name):
    text = re.sub(r"//[^\n]*", "", (CSRC / name).read_text())
    kernels = re.findall(r"__global__.*?\{(.*?)\n\}", text, re.S)
    assert kernels
    for body in kernels:
        wait = min(body.index(w) for w in ("begin_dependent()", "wait_for_previous_kernel()") if w in body)
        before = body[:wait]
        assert "p.seq_lens[" not in before and "*reinterpret_cast" not in before and "atomic" not in before


def test_calls_refuse_null():
    lib = da.load(build_if_missing=True)
    norm, verify = da.NormArgs(), da.VerifyArgs()
    args = da.AppendArgs()
    assert lib.decode_attn_append_normed(None, ctypes.byref(args), ctypes.byref(norm), None, 0, None) == da.DA_ERR_INVALID_ARG
    assert lib.decode_attn_append_normed(None, ctypes.byref(args), None, None, 0, None) == da.DA_ERR_INVALID_ARG
    assert lib.decode_attn_verify(None, ctypes.byref(verify), None, 0, None) == da.DA_ERR_INVALID_ARG
    assert lib.decode_attn_verify(None, None, None, 0, None) == da.DA_ERR_INVALID_ARG


def test_sizes_of_the_argument_structures(tmp_path):
    """The binding's structures are the header's."""
    import subprocess
    src = tmp_path / "sizes.c"
    names = {"da_problem": da.Problem, "da_args": da.Args, "da_append_args": da.AppendArgs, "da_norm_args": da.NormArgs,
             "da_verify_args": da.VerifyArgs, "da_table_args": da.TableArgs, "da_gather_args": da.GatherArgs}
    src.write_text('#include <stdio.h>\n#include "decode_attn.h"\nint main(void) {\n'
                   + "".join(f'printf("%zu\\n", sizeof({n}));\n' for n in names) + "return 0; }\n")
    exe = tmp_path / "sizes"
    include = CSRC.parent.parent / "include"
    subprocess.run(["gcc", "-std=c99", "-I", str(include), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(c) for c in names.values()]
