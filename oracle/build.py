"""Build the C step oracle (test infrastructure) into oracle/libzs_oracle.so,
and the comparison of the library's device arithmetic with its definitions into
oracle/libzs_forms.so.

The oracle is plain C, -O2, no FMA contraction, no fast-math, no flush-to-zero,
so that every fp32 statement of it is one IEEE operation rounded to nearest.
The comparison is compiled as the library is.
"""

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "zs_oracle.c")
LIB = os.path.join(HERE, "libzs_oracle.so")
FORMS = os.path.join(HERE, "libzs_forms.so")


def build(verbose: bool = False) -> str:
    cmd = ["gcc", "-O2", "-std=c11", "-ffp-contract=off", "-fno-fast-math",
           "-fPIC", "-shared", "-Wall", "-Wextra", SRC, "-o", LIB + ".tmp",
           "-lm"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


def build_forms(verbose: bool = False) -> str:
    from zero_sharded_optimizer_shard_amd.build import HIP_FLAGS
    cmd = ["hipcc", *HIP_FLAGS, "-shared", os.path.join(HERE, "forms.hip"),
           "-o", FORMS + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(FORMS + ".tmp", FORMS)
    return FORMS


if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(HERE))
    build(verbose="-v" in sys.argv)
    build_forms(verbose="-v" in sys.argv)
