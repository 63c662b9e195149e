"""The arithmetic by which the 8-bit decode's CTAs share the keys, built for the host from the kernels' own
header."""
from __future__ import annotations

import ctypes
import functools
import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "attention_forward_blackwell_gb300", "csrc")


@functools.lru_cache
def lib():
    with tempfile.TemporaryDirectory() as d:
        path = os.path.join(d, "libq8_line.so")
        subprocess.check_call([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-Wall", "-Werror", "-fPIC",
                               "-shared", "-x", "c++", "-I", CSRC, os.path.join(HERE, "q8_line_walk.cpp"), "-o", path])
        so = ctypes.CDLL(path)
    so.line_levels.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_double, ctypes.c_int]
    return so


def joined(spans, units, block, chunk, splits):
    """0 where every block of every unit has one split and no CTA asks for queries of a unit that is not there."""
    return lib().walk_joined((ctypes.c_int * len(spans))(*spans), len(spans), units, block, chunk, splits)


def line(spans, units, block, slots, levels):
    """(0 where every block has one piece and the merge finds them all, cut: all, big, small, aligned, share)."""
    cut = (ctypes.c_int * 5)()
    bad = lib().walk_line((ctypes.c_int * len(spans))(*spans), len(spans), units, block, slots, levels, cut)
    return bad, dict(zip(("all", "big", "small", "aligned", "share"), cut))
