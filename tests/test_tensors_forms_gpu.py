"""The arithmetic of csrc/zs_codes.h on the GPU, for every input of the ranges
that its comments state: conversion to bf16, roots, a block's quotient, the
codes of m and of roots of v, and the error of the hardware's root that the
codes rely on.  oracle/forms.hip calls the library's own device functions,
compiled as the library is."""

import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import build as ob

pytestmark = pytest.mark.gpu


def floats(lo, hi):
    """How many fp32 numbers are in [lo, hi), 0 <= lo."""
    a, b = (int(np.float32(x).view(np.uint32)) for x in (lo, hi))
    return b - a


def top(q):
    """The first number behind the range of codes up to q."""
    return np.nextafter(np.float32(q * q) * np.float32(1 + 2.0 ** -20),
                        np.float32(np.inf))


@pytest.mark.parametrize("what,name,count", [
    (0, "bf16", 1 << 32),
    (1, "roots", floats(2.0 ** -96, np.inf)),
    (2, "quotients", floats(2.0 ** -100, 2.0 ** 126)),
    # zeros of both signs
    (3, "codes", floats(0, top(127)) + 1 + floats(2.0 ** -123, top(255)) + 2),
    (4, "the hardware's root", floats(0, 65536.0) + 1)])
def test_every_input(what, name, count):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if not os.path.exists(ob.FORMS):
        pytest.fail("libzs_forms.so is not built (run "
                    "__graft_entry__.build())")
    L = ctypes.CDLL(ob.FORMS)
    L.zs_forms_compare.argtypes = [ctypes.c_int, ctypes.c_void_p,
                                   ctypes.c_void_p]
    out = torch.tensor([0, 0, -1], dtype=torch.int64, device="cuda")
    rc = L.zs_forms_compare(what, out.data_ptr(),
                            torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    compared, wrong, first = out.tolist()
    assert wrong == 0, f"{name}: {wrong} inputs, the first {first:#010x}"
    assert compared == count
