"""Which kernels the GPU tests of the Newton-Schulz products run, by the
library's own plan, and that the bounds of full precision would notice a
product with a part missing."""

import shutil

import numpy as np
import pytest

import muon_plan as P
from muon_bounds import full_bound, rel
from oracle import muon as OM


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    return P.build(str(tmp_path_factory.mktemp("plan")))


def test_gpu_tests_run_every_kernel(lib):
    """A new estimate that sends these stacks to other kernels shows here."""
    seen = set()
    for (precision, last), stacks in P.COVER.items():
        for s in stacks:
            seen |= P.kernels(lib, s, precision, last)
    want = set()
    for precision in ("fast", "full"):
        for t in P.TILES:
            want |= {(precision, e, t) for e in (P.POLY, P.PROD)}
            for tall in (False, True):
                want |= {(precision, e, t, tall) for e in (P.GRAM, P.UPDATE)}
                want |= {(precision, e, t, tall, by4)
                         for e in (P.OUT_BF16, P.OUT_F32, P.STEP)
                         for by4 in (False, True)}
    assert len(want) == 144
    assert seen == want


def test_plan_of_a_call(lib):
    """Five steps of three products one by one; with the first two together
    four rounds, of which the first has two polynomials and three products
    of squares; nothing for small matrices."""
    one = P.launches(lib, [(1, 512, 520)], P.OUT_F32, False)
    assert [e for e, _, _ in one] == [P.GRAM, P.POLY, P.UPDATE] * 4 + [
        P.GRAM, P.POLY, P.OUT_F32]
    two = P.launches(lib, [(24, 256, 3000)], P.STEP, False)
    first = [P.GRAM] + [P.POLY] * 2 + [P.PROD] * 3 + [P.UPDATE]
    assert [e for e, _, _ in two] == first + [P.GRAM, P.POLY, P.UPDATE] * 2 + [
        P.GRAM, P.POLY, P.STEP]
    full = P.launches(lib, [(24, 256, 3000)], P.STEP, True)
    assert [e for e, _, _ in full] == first + [P.GRAM, P.POLY, P.UPDATE] + \
        first[:-1] + [P.STEP]
    assert P.launches(lib, [(9, 64, 500), (1, 128, 100)], P.STEP, False) == []
    # coefficients whose product leaves fp16's range
    big = P.launches(lib, [(24, 256, 3000)], P.STEP, False, coef=(5., -8., 4.))
    assert P.PROD not in [e for e, _, _ in big]


def test_few_rows_by_themselves(lib):
    """Beside stacks that take twos, in launches of their own and one by one;
    by themselves one by one."""
    stacks = [(1, 8, 6000), (8, 256, 8000), (1, 6000, 3)]
    got = P.launches(lib, stacks, P.OUT_F32, False)
    assert {p for _, _, p in got} == {0, 1}
    assert P.PROD not in [e for e, _, p in got if p == 0]
    assert P.PROD in [e for e, _, p in got if p == 1]
    assert P.PROD not in [e for e, _, _ in P.launches(
        lib, stacks[:1], P.OUT_F32, False)]


@pytest.mark.parametrize("rows,twos", [(1, True), (2, False), (63, False),
                                       (64, False), (127, False),
                                       (128, True), (192, True)])
def test_rows_from_which_steps_go_together(lib, rows, twos):
    """In fast precision; in full precision all of them do."""
    for r, c in ((rows, 8000), (8000, rows)):
        got = P.launches(lib, [(60, r, c)], P.OUT_F32, False)
        assert (P.PROD in [e for e, _, _ in got]) == twos
        got = P.launches(lib, [(60, r, c)], P.OUT_F32, True)
        assert P.PROD in [e for e, _, _ in got]


# shorter side first, where twos are likely and where they are not
@pytest.mark.parametrize("shape", [(65, 69), (66, 275), (136, 588), (157, 1230),
                                   (204, 545), (399, 403), (333, 1001)],
                         ids=lambda s: "%dx%d" % s)
def test_full_bounds_notice_a_missing_part(shape):
    """Each product of full precision without its high x low or low x high
    part is at least twice the bound off."""
    U = np.random.default_rng(5).standard_normal(shape)
    e = OM.orthogonalize(U)
    t = full_bound(U, e)
    for pairs in (False, True):
        for what in ("gram", "poly", "prod", "update"):
            for part in ("hl", "lh"):
                if what == "prod" and not pairs:
                    continue
                off = rel(OM.rounded(U, full=True, pairs=pairs,
                                     drop=(what, part)), e)
                assert off > 2 * t, (pairs, what, part, off, t)
