"""zs_muon.h without a GPU: every declared symbol is there, argument checks
return the documented codes before any device work, workspaces grow as
documented; and the float64 oracle of the Muon operators against singular
values and against itself."""

import ctypes
import os
import re

import numpy as np
import pytest

import zero_sharded_optimizer_shard_amd as zs
from oracle import muon as OM
from zero_sharded_optimizer_shard_amd import _muon as zm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EALIGN, ERANGE = -1, -2, -3
F = ctypes.c_float
GOOD = 1 << 20          # an address that is never touched: calls that reach
                        # the device are not made here


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "zs_muon.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = sorted(set(re.findall(r"\b(zs_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(zs.MUON_EXPORTS)
    for n in names:
        assert hasattr(zs.lib(), n)


def test_header_is_plain_c(tmp_path):
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("gcc not found")
    c = tmp_path / "a.c"
    c.write_text('#include "zs_muon.h"\n'
                 'int sizes(void) { return (int)(sizeof(zs_muon) + '
                 'sizeof(zs_muon_tensor) + sizeof(zs_ns_matrices)); }\n')
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "include"), "-c", str(c), "-o",
                    str(tmp_path / "a.o")], check=True)


def ns(steps=5, precision=0, eps=1e-7, coef=OM.COEF):
    s = zm.zs_newton_schulz(steps, precision, eps)
    for k in range(zs.ZS_NS_MAX_STEPS):
        s.coef[k] = (F * 3)(*coef)
    return s


def mats(n=1, **kw):
    a = (zm.zs_ns_matrices * n)()
    for m in a:
        m.x, m.o, m.batch, m.rows, m.cols = GOOD, 2 * GOOD, 2, 8, 16
        m.x_batch_stride, m.x_row_stride = 128, 16
        m.o_batch_stride, m.o_row_stride = 128, 16
        for k, v in kw.items():
            setattr(m, k, v)
    return a


def orth(count=1, m=None, xt=0, ot=0, s=None, ws=GOOD, nbytes=1 << 40):
    return zm._lib().zs_orthogonalize(
        count, mats(max(count, 1)) if m is None else m, xt, ot,
        ctypes.byref(ns() if s is None else s), ws, nbytes, None)


@pytest.mark.parametrize("code,kw", [
    (EINVAL, dict(count=0)), (EINVAL, dict(count=17)),
    (EINVAL, dict(xt=2)), (EINVAL, dict(ot=-1)),
    (EINVAL, dict(s=ns(steps=0))), (EINVAL, dict(s=ns(steps=17))),
    (EINVAL, dict(s=ns(precision=2))), (EINVAL, dict(s=ns(eps=0))),
    (EINVAL, dict(s=ns(eps=-1))), (EINVAL, dict(s=ns(eps=float("inf")))),
    (EINVAL, dict(s=ns(eps=float("nan")))),
    (EINVAL, dict(s=ns(coef=(1, float("nan"), 0)))),
    (EINVAL, dict(s=ns(coef=(float("inf"), 1, 0)))),
    (EINVAL, dict(ws=None)), (EALIGN, dict(ws=GOOD + 128)),
    (ERANGE, dict(nbytes=1000)), (ERANGE, dict(nbytes=-1)),
    (EINVAL, dict(m=mats(x=None))), (EINVAL, dict(m=mats(o=None))),
    (EALIGN, dict(m=mats(x=GOOD + 1))), (EALIGN, dict(m=mats(o=GOOD + 1))),
    (EALIGN, dict(m=mats(x=GOOD + 2), xt=1)),
    (EALIGN, dict(m=mats(o=GOOD + 2), ot=1)),
    (EINVAL, dict(m=mats(batch=-1))), (EINVAL, dict(m=mats(rows=-1))),
    (EINVAL, dict(m=mats(cols=-5))),
    (EINVAL, dict(m=mats(x_row_stride=15))),
    (EINVAL, dict(m=mats(o_row_stride=15))),
    (EINVAL, dict(m=mats(o_row_stride=0))),
    (EINVAL, dict(m=mats(x_batch_stride=-1))),
    (EINVAL, dict(m=mats(o_batch_stride=127))),
    (EINVAL, dict(m=mats(o_batch_stride=0))),
    (ERANGE, dict(m=mats(x_row_stride=1 << 60))),
    (ERANGE, dict(m=mats(x_batch_stride=1 << 62))),
    (ERANGE, dict(m=mats(o_row_stride=1 << 62))),
    (ERANGE, dict(m=mats(o_batch_stride=1 << 62))),
    (ERANGE, dict(m=mats(rows=1 << 40, cols=1 << 40))),
    (ERANGE, dict(m=mats(rows=65536, cols=65536))),
    (ERANGE, dict(m=mats(rows=40000, cols=40000))),
    (ERANGE, dict(m=mats(rows=1, cols=(1 << 22) + 1))),
    (ERANGE, dict(m=mats(batch=1 << 40))),
    (ERANGE, dict(m=mats(batch=(1 << 23) + 1, rows=1, cols=1)))])
def test_orthogonalize_refusals(code, kw):
    assert orth(**kw) == code
    assert zs.zs_last_error()


def test_orthogonalize_null_structs():
    L = zm._lib()
    assert L.zs_orthogonalize(1, None, 0, 0, ctypes.byref(ns()), GOOD,
                              1 << 40, None) == EINVAL
    assert L.zs_orthogonalize(1, mats(), 0, 0, None, GOOD, 1 << 40,
                              None) == EINVAL
    b = ctypes.c_int64()
    assert L.zs_orthogonalize_workspace(1, None, 0,
                                        ctypes.byref(b)) == EINVAL
    assert L.zs_orthogonalize_workspace(1, mats(), 0, None) == EINVAL
    assert L.zs_orthogonalize_workspace(0, mats(), 0,
                                        ctypes.byref(b)) == EINVAL
    assert L.zs_orthogonalize_workspace(1, mats(), 5,
                                        ctypes.byref(b)) == EINVAL


@pytest.mark.parametrize("empty", [dict(batch=0), dict(rows=0),
                                   dict(cols=0)])
def test_nothing_to_do_touches_nothing(empty):
    m = mats(x=None, o=None, **empty)
    assert orth(m=m, ws=None, nbytes=0) == 0


def test_workspace_sizes():
    def need(precision, *shapes):
        a = mats(len(shapes))
        for m, (b, r, c) in zip(a, shapes):
            m.batch, m.rows, m.cols = b, r, c
        out = ctypes.c_int64()
        assert zm._lib().zs_orthogonalize_workspace(
            len(shapes), a, precision, ctypes.byref(out)) == 0
        return out.value

    one = need(0, (1, 100, 200))
    # X in both orientations, twice, A and B, on sides rounded up to 64
    assert 12 * 128 * 256 + 4 * 128 * 128 <= one < 2 * 12 * 128 * 256
    assert need(0, (1, 200, 100)) == one
    assert need(1, (1, 100, 200)) > one
    assert need(0, (1, 100, 200), (1, 100, 200), (0, 5, 5)) == 2 * one
    assert need(0, (0, 5, 5)) == 0
    # past 32 bits
    assert need(0, (100, 4096, 14336)) > 12 * 100 * 4096 * 14336 > 1 << 32
    assert orth(m=mats(), nbytes=need(0, (2, 8, 16)) - 1) == ERANGE


def test_outputs_side_by_side():
    """Two matrices of 8 x 16 in rows of their own, or overlapping by one
    element; past the strides the first lacks its workspace."""
    for batch, row, code in ((16, 32, ERANGE), (16, 31, EINVAL),
                             (15, 32, EINVAL), (20, 36, ERANGE),
                             (20, 35, EINVAL)):
        m = mats(o_batch_stride=batch, o_row_stride=row)
        assert orth(m=m, nbytes=0) == code


@pytest.mark.parametrize("precision", [0, 1])
def test_largest_call(precision):
    """A launch has fewer than 2^32 threads, and a matrix of one tile up to
    512: 2^23 of them are refused by the call and by its workspace, one less
    is not."""
    a = mats(batch=1 << 23, rows=1, cols=1, x_batch_stride=1,
             o_batch_stride=1, x_row_stride=1, o_row_stride=1)
    b = ctypes.c_int64()
    assert orth(m=a, s=ns(precision=precision)) == ERANGE
    size = zm._lib().zs_orthogonalize_workspace
    assert size(1, a, precision, ctypes.byref(b)) == ERANGE
    a[0].batch -= 1
    assert size(1, a, precision, ctypes.byref(b)) == 0
    # the same over two stacks
    two = mats(2, batch=1 << 22, rows=1, cols=1)
    assert size(2, two, precision, ctypes.byref(b)) == ERANGE
    lay = zs.zs_layout_build_tensors([1 << 23], 1, 0)
    assert step(lay=lay, t=((0, 1 << 23, 1, 1),),
                hp=muon(ns=ns(precision=precision))) == ERANGE


def layout():
    return zs.zs_layout_build_tensors([64 * 48, 300, 5 * 7], 1, 0)


def muon(**kw):
    hp = zm.zs_muon(1e-3, 0.95, 0.1, 1, 2, ns())
    for k, v in kw.items():
        setattr(hp, k, v)
    return hp


def step(lay=None, count=1, t=((0, 1, 64, 48),), grads=GOOD, gl=1, gs=0,
         state=GOOD, shard=GOOD, flat=GOOD, hp=None, ws=GOOD,
         nbytes=1 << 40):
    lay = lay or layout()
    arr = (zm.zs_muon_tensor * max(len(t), 1))(
        *[zm.zs_muon_tensor(*x) for x in t])
    g = (ctypes.c_void_p * max(len(t), 1))(*[grads] * len(t))
    return zm._lib().zs_muon_step(
        lay.handle, count, arr, g, gl, gs, state, shard, flat,
        ctypes.byref(hp or muon()), ws, nbytes, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("code,kw", [
    (EINVAL, dict(count=0)), (EINVAL, dict(count=17)),
    (ERANGE, dict(t=((3, 1, 64, 48),))), (ERANGE, dict(t=((-1, 1, 64, 48),))),
    (EINVAL, dict(count=2, t=((0, 1, 64, 48), (0, 1, 64, 48)))),
    (EINVAL, dict(t=((0, 1, 64, 47),))), (EINVAL, dict(t=((0, 2, 64, 48),))),
    (EINVAL, dict(t=((0, 0, 64, 48),))), (EINVAL, dict(t=((0, 1, -64, 48),))),
    (ERANGE, dict(t=((0, 1, 1 << 40, 1 << 40),))),
    (EINVAL, dict(gl=2)), (EINVAL, dict(grads=None)),
    (EALIGN, dict(grads=GOOD + 8)), (EALIGN, dict(gl=0, gs=3073)),
    (ERANGE, dict(gl=0, gs=64 * 48 - 8)), (ERANGE, dict(gl=0, gs=-8)),
    (ERANGE, dict(gl=0, gs=(2**63 - 8))),
    (EINVAL, dict(state=None)), (EALIGN, dict(state=GOOD + 8)),
    (EINVAL, dict(shard=None, flat=None)),
    (EALIGN, dict(shard=GOOD + 2)), (EALIGN, dict(flat=GOOD + 8)),
    (EINVAL, dict(ws=None)), (EALIGN, dict(ws=GOOD + 16)),
    (ERANGE, dict(nbytes=4096)),
    (EINVAL, dict(hp=muon(lr=NAN))), (EINVAL, dict(hp=muon(momentum=INF))),
    (EINVAL, dict(hp=muon(weight_decay=NAN))), (EINVAL, dict(hp=muon(scale=3))),
    (EINVAL, dict(hp=muon(scale=-1))), (EINVAL, dict(hp=muon(ns=ns(steps=0)))),
    (EINVAL, dict(hp=muon(ns=ns(eps=0))))])
def test_step_refusals(code, kw):
    if kw.get("gs") == 2**63 - 8:       # overflows only with several ranks
        kw = dict(kw, lay=zs.zs_layout_build_tensors([64 * 48] * 3, 3, 0))
    assert step(**kw) == code
    assert zs.zs_last_error()


@pytest.mark.parametrize("hp", [
    dict(lr=3e38), dict(lr=-3e38), dict(lr=1e30, weight_decay=1e10, scale=0),
    dict(lr=1e30, weight_decay=-1e10, scale=0)])
def test_step_refuses_factors_that_overflow(hp):
    """lr is finite, lr * 0.2 * sqrt(64) and 1 - lr * weight_decay are not:
    they would make NaN of a weight whose update is zero."""
    assert step(hp=muon(**hp)) == EINVAL
    assert "finite" in zs.zs_last_error()


def test_step_needs_a_whole_tensor_layout():
    lay = zs.zs_layout_build([64 * 48], 1, 0)
    assert step(lay=lay) == EINVAL
    with pytest.raises(zs.ZsError):
        zs.zs_muon_workspace(lay, [(0, 64, 48)])


def test_step_null_structs():
    L, lay, b = zm._lib(), layout(), ctypes.c_int64()
    t = (zm.zs_muon_tensor * 1)(zm.zs_muon_tensor(0, 1, 64, 48))
    g = (ctypes.c_void_p * 1)(GOOD)
    tail = (GOOD, GOOD, GOOD)

    def call(lay_h, t, g, hp):
        return L.zs_muon_step(lay_h, 1, t, g, 1, 0, *tail, hp, GOOD, 1 << 40,
                              None)
    assert call(None, t, g, ctypes.byref(muon())) == EINVAL
    assert call(lay.handle, None, g, ctypes.byref(muon())) == EINVAL
    assert call(lay.handle, t, None, ctypes.byref(muon())) == EINVAL
    assert call(lay.handle, t, g, None) == EINVAL
    assert L.zs_muon_workspace(None, 1, t, 0, ctypes.byref(b)) == EINVAL
    assert L.zs_muon_workspace(lay.handle, 1, None, 0,
                               ctypes.byref(b)) == EINVAL
    assert L.zs_muon_workspace(lay.handle, 1, t, 0, None) == EINVAL
    assert L.zs_muon_workspace(lay.handle, 1, t, 9,
                               ctypes.byref(b)) == EINVAL


def test_binding_refuses_before_the_library():
    import torch
    x = torch.zeros(4, 4)
    kw = dict(workspace=torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError):         # host tensors
        zs.zs_orthogonalize([x], [x], **kw)
    with pytest.raises(ValueError):
        zs.zs_orthogonalize([x], [], **kw)
    with pytest.raises(ValueError):
        zs.zs_orthogonalize_workspace([torch.zeros(4)])
    with pytest.raises(ValueError):         # columns not contiguous
        zs.zs_orthogonalize_workspace([torch.zeros(4, 6).t()])
    with pytest.raises(ValueError):
        zs.zs_muon_workspace(layout(), [(0, 64)])
    with pytest.raises(ValueError):
        zm._newton_schulz(3, [OM.COEF] * 2, 1e-7, "fast")
    with pytest.raises(ValueError):
        zs.zs_muon_step(layout(), [(0, 64, 48)], [x], x, lr=1., momentum=0.,
                        weight_decay=0., **kw)


@pytest.mark.parametrize("coef", [(), (3.4, -4.8), (1., 2., 3., 4.),
                                  [(1., 2., 3.), (1., 2.)]],
                         ids=["none", "two", "four", "short row"])
def test_binding_refuses_coefficients(coef):
    with pytest.raises(ValueError):
        zm._newton_schulz(2, coef, 1e-7, "fast")


def test_binding_refuses_integers_that_do_not_fit():
    """2^32 is 0 to a 32-bit field: another tensor, another precision."""
    big = 1 << 32
    for t in ((big, 64, 48), (0, (1 << 64) + 64, 48), (-big, 1, 64, 48)):
        with pytest.raises(ValueError):
            zs.zs_muon_workspace(layout(), [t])
    with pytest.raises(ValueError):
        zs.zs_muon_workspace(layout(), [(0, 64, 48)], precision=big)
    for steps in (big + 5, -big + 5, 1 << 70):
        with pytest.raises(ValueError):
            zm._newton_schulz(steps, OM.COEF, 1e-7, "fast")
    with pytest.raises(ValueError):
        zm._newton_schulz(5, OM.COEF, 1e-7, big + 1)
    with pytest.raises(TypeError):
        zm._newton_schulz(5.0, OM.COEF, 1e-7, "fast")
    # in 32 bits, and the library's to refuse
    assert zm._newton_schulz(1 << 30, OM.COEF, 1e-7, "fast").steps == 1 << 30
    assert zm._newton_schulz(np.int64(3), OM.COEF, 1e-7, "full").steps == 3
    assert zs.zs_muon_workspace(layout(), [(np.int64(0), 64, 48)]) > 0


# ---- the oracle -------------------------------------------------------------

@pytest.mark.parametrize("shape", [(20, 33), (33, 20), (24, 24), (1, 9)])
def test_oracle_maps_singular_values(shape):
    U = np.random.default_rng(1).standard_normal(shape)
    eps = 1e-7
    u, s, vt = np.linalg.svd(U, full_matrices=False)
    s = s / (np.sqrt(np.sum(U * U)) + np.float64(np.float32(eps)))
    for _ in range(5):
        a, b, c = OM.COEF
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(OM.orthogonalize(U, 5, OM.COEF, eps), (u * s) @ vt,
                       rtol=0, atol=1e-11)


def directions(kind, rng, m, n):
    """`kind` 8: eight directions 100 times the others; k: singular values
    1/k."""
    def q(a, b):
        return np.linalg.qr(rng.standard_normal((a, b)))[0]
    if kind == "k":
        return (q(m, m) / np.arange(1, m + 1.)) @ q(n, m).T
    w = rng.standard_normal((m, n))
    return w / np.linalg.norm(w, 2) + 100 * q(m, 8) @ q(n, 8).T


@pytest.mark.parametrize("steps", [5, 6, 10])
@pytest.mark.parametrize("kind", ["8", "k"])
def test_steps_together_cost_no_accuracy(kind, steps):
    """In fast precision: another draw of roundings as large, so at most
    twice those of steps one by one."""
    U = directions(kind, np.random.default_rng(3), 256, 1061)
    e = OM.orthogonalize(U, steps)
    one, two = (np.linalg.norm(OM.rounded(U, steps, pairs=p) - e)
                for p in (False, True))
    assert two <= 2 * one


@pytest.mark.parametrize("full,u", [(False, 2.0 ** -11), (True, 2.0 ** -22)])
@pytest.mark.parametrize("shape", [(40, 90), (90, 40), (64, 64)])
def test_rounded_oracle_of_one_step(shape, full, u):
    """One step from |X|_F = 1, every rounding off by u at most: A by 3u (its
    two operands and itself), B by (|b| + 2c) 3u + (|b| + c) u, and B X by
    that and by max |b s + c s^2| u = 2.8u: under 37u in all."""
    rng = np.random.default_rng(2)
    for U in (rng.standard_normal(shape),
              rng.standard_normal((shape[0], 3)) @
              rng.standard_normal((3, shape[1]))):
        e = OM.orthogonalize(U, 1)
        r = OM.rounded(U, 1, full=full)
        d = np.linalg.norm(r - e)
        assert 0 < d <= 37 * u
        # over five steps, full precision's eleven bits more are there
        d5 = [np.linalg.norm(OM.rounded(U, full=f) - OM.orthogonalize(U))
              for f in (False, True)]
        assert d5[1] < d5[0] / 2 ** 8


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("size", [1e-8, 1e-10, 1e-14, 1e-20])
def test_norms_below_eps_keep_their_bits(size, full):
    """A matrix far below eps stays as exact as its representation: the steps
    multiply it by a and little else."""
    U = np.random.default_rng(4).standard_normal((64, 256))
    U *= size / np.linalg.norm(U)
    for steps in (5, 10):
        e = OM.orthogonalize(U, steps)
        r = OM.rounded(U, steps, full=full)
        off = np.linalg.norm(r - e) / np.linalg.norm(e)
        # where singular values have come near one, roundings are fast's own
        big = np.linalg.norm(e) > 0.1
        assert off <= (2e-3 if big and not full else 1e-6)
