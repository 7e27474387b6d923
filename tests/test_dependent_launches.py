"""Kernels that are launched as dependents (launch_after) may start while the kernel before them still runs.  What
an earlier kernel wrote is theirs to see only after the wait, so each of them waits before it looks at any memory."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "packed_varlen_attention_cu_gb300", "csrc")


def sources():
    text = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path, encoding="utf-8") as f:
            text[os.path.basename(path)] = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    return text


def kernels(text):
    """Names and bodies of the kernels of a file."""
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^)]*\)\s*)?(\w+)\s*\(", text):
        at = text.index("{", m.end())
        depth, end = 1, at + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        yield m.group(1), text[at + 1:end - 1]


def dependents():
    """(file, kernel) of all that launch_after is given, by name or by a variable that holds the name."""
    found = set()
    for name, text in sources().items():
        for arg in re.findall(r"launch_after\(\s*(\w+)", text):
            held = re.findall(r"auto\s+%s\s*=\s*([^;]*);" % arg, text)
            for kernel in re.findall(r"\w+_kernel", " ".join(held)) if held else [arg]:
                found.add((name, kernel))
    return sorted(found - {("launch.cuh", "void")})


def test_all_dependents_are_found():
    names = {k for _, k in dependents()}
    assert {"bwd_dq_kernel", "bwd_dkdv_kernel", "scan_kernel", "move_kernel", "rows_kernel", "attn_kernel", "join_kernel"} <= names


@pytest.mark.parametrize("file,kernel", dependents())
def test_it_waits_before_it_reads(file, kernel):
    every = sources()
    bodies = [b for text in [every[file]] + [t for n, t in every.items() if n.endswith("cuh")] for k, b in kernels(text) if k == kernel]
    assert bodies
    for body in bodies:
        before, wait, _ = body.partition("wait_previous();")
        assert wait
        # the wait is every thread's, and nothing before it goes through a pointer
        assert before.count("{") == before.count("}")
        before = re.sub(r"&\w+->\w+", "", before)  # (addresses of fields)
        assert not re.search(r"->|\bif\b|\bfor\b|\bwhile\b|\breturn\b|\bstruct\b|\bld\.|__ldg|cp_async|load\w*\(", before), before
