"""Which kernels a Newton-Schulz call launches, by the library's own plan
(csrc/zs_muon_plan.h, built with g++ into a library beside the tests' other
files of a run), and the stacks that the GPU tests take so that every kernel
of the products is run.  TEST INFRASTRUCTURE."""

import ctypes
import os
import subprocess

from oracle import muon as OM
from zero_sharded_optimizer_shard_amd import _muon as zm

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
GRAM, POLY, PROD, UPDATE, OUT_BF16, OUT_F32, STEP = range(7)
TILES = (64, 128, 192, 256)


def build(path):
    so = os.path.join(path, "libmuon_plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fPIC",
                    "-shared", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "zero_sharded_optimizer_shard_amd",
                                 "csrc"),
                    os.path.join(HERE, "muon_plan.cpp"), "-o", so],
                   check=True, capture_output=True, text=True)
    return ctypes.CDLL(so)


def launches(lib, stacks, last, full, steps=5, coef=OM.COEF):
    """[(product, tile, part)] of a call on stacks [(batch, rows, cols)]."""
    ns = zm._newton_schulz(steps, coef, 1e-7, "full" if full else "fast")
    n = len(stacks)
    sizes = (ctypes.c_int64 * (3 * n))(*[v for s in stacks for v in s])
    rec = (ctypes.c_int32 * 3000)()
    got = lib.muon_plan(n, sizes, last, ctypes.byref(ns), rec, 1000)
    assert got >= 0
    return [tuple(rec[3 * k:3 * k + 3]) for k in range(got)]


# Stacks (batch, rows, cols) by precision and last update: between them they
# run every product by every tile, wide and tall where the operands depend on
# it, and every last update also by fours and one by one (columns a multiple
# of four or not).  No side is a multiple of a tile.
COVER = {
    ('fast', OUT_BF16): [(1, 65, 139), (1, 68, 144), (1, 135, 65), (1, 136,
        68), (36, 67, 473), (36, 68, 456), (36, 140, 936), (36, 504, 72), (36,
        904, 129), (36, 940, 132), (60, 135, 539), (60, 136, 860), (60, 155,
        815), (60, 274, 67), (60, 803, 135), (60, 820, 140)],
    ('fast', OUT_F32): [(1, 66, 155), (1, 68, 132), (1, 160, 68), (1, 170,
        65), (36, 129, 931), (36, 519, 680), (36, 948, 132), (60, 72, 296),
        (60, 132, 960), (60, 145, 803), (60, 259, 73), (60, 320, 68), (60,
        391, 619), (60, 547, 129), (60, 772, 136), (60, 860, 133)],
    ('fast', STEP): [(1, 67, 136), (9, 137, 1502), (1, 1771, 5880), (1, 1869, 5502), (1, 6097,
        1675), (1, 6860, 1680), (24, 652, 84), (36, 292, 267), (36, 610, 521),
        (60, 73, 523), (60, 93, 564), (60, 148, 740), (60, 152, 726), (60,
        194, 519), (60, 432, 392), (60, 730, 153), (60, 740, 136)],
    ('full', OUT_BF16): [(1, 67, 75), (1, 68, 68), (1, 72, 65), (1, 88, 68),
        (36, 76, 522), (36, 904, 132), (60, 68, 324), (60, 136, 588), (60,
        145, 539), (60, 148, 780), (60, 204, 545), (60, 264, 72), (60, 275,
        66), (60, 531, 195), (60, 605, 137), (60, 788, 144)],
    ('full', OUT_F32): [(1, 66, 68), (1, 72, 66), (1, 76, 68), (1, 157, 1230),
        (36, 133, 1007), (36, 532, 664), (36, 599, 521), (36, 916, 140), (60,
        67, 267), (60, 132, 872), (60, 136, 787), (60, 390, 576), (60, 404,
        68), (60, 561, 131), (60, 888, 136), (60, 912, 135)],
    ('full', STEP): [(1, 65, 69), (1, 68, 72), (1, 75, 66), (1, 76, 72), (5,
        3696, 577), (9, 1892, 588), (16, 580, 1072), (24, 587, 662), (36, 136,
        933), (60, 72, 524), (60, 81, 522), (60, 140, 548), (60, 403, 399),
        (60, 532, 72), (60, 544, 136), (60, 661, 129)],
}


def kernels(lib, stack, precision, last):
    """What a call on one stack runs, as (product, tile, and what else its
    kernel's work depends on)."""
    _, r, c = stack
    out = set()
    for e, t, _ in launches(lib, [stack], last, precision == "full"):
        how = () if e in (POLY, PROD) else (r > c,)
        if e >= OUT_BF16:
            how += (c % 4 == 0,)
        out.add((precision, e, t) + how)
    return out
