"""Copies of the library for the tests of attention of requests that share a prefix: how
groups are read (each request for itself, in groups, together) is set by the test instead
of by the sizes; with giving_up, warps also give up on one of their first pieces of the
cache."""
import contextlib
import ctypes
import functools
import os
import tempfile

from bitwise_reproducible_fp32_gb300 import build, detlib

ALONE, GROUPS, TOGETHER = 0, 1, 2
RINGS = ["decode.cu", "decode_shared.cu", "decode_few.cu", "decode_group.cu"]


@functools.cache
def library(giving_up=False):
    out = os.path.join(tempfile.mkdtemp(prefix="detfp32_"), "libdetfp32_variant.so")
    if giving_up:
        build.build_variant(["DET_TEST_SHARED_HOW", "DET_TEST_DECODE_GIVE_UP"], out, RINGS)
    else:
        build.build_variant(["DET_TEST_SHARED_HOW"], out, ["decode_shared.cu"])
    lib = ctypes.CDLL(out)
    for name, res, args in detlib.SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


@contextlib.contextmanager
def reading(how, giving_up=False):
    """The binding's calls go to that copy, which reads every group of two or more requests
    so (in groups: those of at most 8 query rows a key-value head, others together)."""
    lib = library(giving_up)
    shipped, sizes = detlib.load(), dict(detlib._decode_workspaces)
    word = ctypes.c_int.in_dll(lib, "det_test_shared_how")
    before, word.value = word.value, how
    detlib._lib = lib
    detlib._decode_workspaces.clear()
    try:
        yield lib
    finally:
        word.value = before
        detlib._lib = shipped
        detlib._decode_workspaces.clear()
        detlib._decode_workspaces.update(sizes)
