"""The argument structs that Python declares, field by field against include/ssu.h as a C compiler
lays them out."""

from __future__ import annotations

import ctypes
import subprocess
from pathlib import Path

import pytest

import selective_state_update_02_gb300 as ssu

ROOT = Path(__file__).resolve().parents[1]
STRUCTS = ["ssu_shape_t", "ssu_strides_t", "ssu_launch_t", "ssu_token_strides_t",
           "ssu_block_tensor_t", "ssu_copy_launch_t", "ssu_rotate_shape_t", "ssu_rotate_strides_t",
           "ssu_attend_shape_t", "ssu_attend_strides_t"]


def declared(cls):
    return [(name, getattr(cls, name).offset, getattr(cls, name).size)
            for name, *_ in cls._fields_]


@pytest.fixture(scope="module")
def header(tmp_path_factory):
    """The header's (field, offset, size) of every struct, for the fields that Python names."""
    tmp = tmp_path_factory.mktemp("layout")
    lines = []
    for s in STRUCTS:
        lines.append(f'printf("{s} . 0 %zu\\n", sizeof({s}));')
        lines += [f'printf("{s} {f} %zu %zu\\n", offsetof({s}, {f}), sizeof((({s} *)0)->{f}));'
                  for f, *_ in getattr(ssu, s)._fields_]
    (tmp / "layout.c").write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ssu.h"\n'
                                  "int main(void) {\n" + "\n".join(lines) + "\nreturn 0;\n}\n")
    subprocess.run(["gcc", "-std=c99", "-I", str(ROOT / "include"), str(tmp / "layout.c"), "-o",
                    str(tmp / "layout")], check=True)
    out = subprocess.run([str(tmp / "layout")], capture_output=True, text=True, check=True).stdout
    found = {s: [] for s in STRUCTS}
    for line in out.splitlines():
        s, field, offset, size = line.split()
        found[s].append((field, int(offset), int(size)))
    return found


@pytest.mark.parametrize("struct", STRUCTS)
def test_python_declares_what_the_header_says(header, struct):
    cls = getattr(ssu, struct)
    (_, _, size), *fields = header[struct]
    assert ctypes.sizeof(cls) == size
    assert declared(cls) == fields
    # no bytes between the declared fields that a field of the header's alone could hide in
    end = 0
    for name, offset, width in declared(cls):
        assert offset == end, name
        end += width
    assert end == size
