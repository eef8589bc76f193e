"""Programmatic dependent launch, checked in the sources: a kernel that is
launched with the attribute has to wait for the previous grid somewhere, or it
may read and overwrite what that grid still uses, and a later kernel's wait
covers only it."""
from __future__ import annotations

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_quantized_packed_gb300", "csrc")


def text(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def matching(s, at, pair):
    """The text from the bracket at `at` to the one that closes it."""
    depth = 0
    for i in range(at, len(s)):
        depth += (s[i] == pair[0]) - (s[i] == pair[1])
        if depth == 0:
            return s[at:i + 1]
    raise AssertionError("unbalanced")


def kernels(s):
    """(name, body) of every __global__ function."""
    for m in re.finditer(r"__global__ void", s):
        at = m.end()
        if s[at:].lstrip().startswith("__launch_bounds__"):
            at = s.index("__launch_bounds__", at)
            at += len("__launch_bounds__")
            at += len(matching(s, at, "()"))
        name = re.match(r"\s*(\w+)\s*\(", s[at:])
        args = at + name.end() - 1
        body = args + len(matching(s, args, "()"))
        yield name.group(1), matching(s, s.index("{", body), "{}")


def launches(s):
    """The argument lists of every call of launch()."""
    for m in re.finditer(r"(?<![\w.])launch\(", s):
        yield matching(s, m.end() - 1, "()")


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))),
                         ids=os.path.basename)
def test_a_kernel_launched_with_pdl_waits(path):
    s = text(path)
    idle = [name for name, body in kernels(s) if "pdl_wait()" not in body]
    for args in launches(s):
        if "pdl" in args:
            assert not [k for k in idle if re.search(rf"\b{k}\b", args)], args
    # Where the attribute is set by hand, every kernel of the file but an empty one is launched so.
    if "ProgrammaticStreamSerialization" in s:
        for name, body in kernels(s):
            assert "pdl_wait()" in body or body.replace(" ", "") == "{}", name
