"""What holding the states in 8 bits costs over thousands of steps, beside fp32
states: the figures that include/zs_tensors.h states, from oracle/tensors.py's
rules on noise with a mean of a tenth of its sigma.

The rules run here over all blocks at once; `test_rules_are_the_oracles` holds
them to oracle/tensors.py bit for bit."""

import numpy as np
import pytest

from oracle import tensors as OT

F = np.float32
BLOCK, NB = OT.BLOCK, 16


def encode(x, top):
    """OT.encode of [NB, BLOCK] values whose blocks are finite."""
    a = np.abs(x)
    A = a.max(1, keepdims=True)
    some = A >= F(2.0 ** -100)
    S = np.where(some, A * F(1 / top ** 2), F(0)).astype(F)
    inv = np.where(some, F(top ** 2) / np.where(some, A, F(1)), F(0))
    y = a * inv.astype(F)
    k = np.floor(np.sqrt(y.astype(np.float64)))
    k += (k + 0.5) ** 2 <= y
    if top == 255:
        k = np.where(some, np.maximum(k, a > 0), k)
    return np.copysign(k, x).astype(F), S, y


def held_m(m, blank):
    """(codes, scales) of m as a step holds them."""
    q, S, y = encode(m, 127)
    live = ~blank.all(1, keepdims=True)
    down = live & blank & (np.abs(q) <= OT.FADE) & (q * q > y)
    return q - np.sign(q) * down, S


def decode(q, S):
    return (q * np.abs(q)) * S


class Training:
    """Steps of lr 1 and no decay with 8-bit states and with fp32 ones over
    the same gradients."""

    def __init__(self, beta1=0.9, beta2=0.95, fade=True):
        self.hp, self.t, self.fade = (1.0, beta1, beta2, 1e-8, 0.0), 0, fade
        z = np.zeros((NB, BLOCK), F)
        s = np.zeros((NB, 1), F)
        self.m, self.v = z, z
        self.q = z, s, z, s
        self.w8, self.w = z.astype(np.float64), z.astype(np.float64)

    def step(self, g):
        self.t += 1
        b1, omb1, b2, omb2, ss, bc2s, _, eps = OT.constants(self.hp, self.t)
        mq, ms, rq, rs = self.q
        r0 = decode(rq, rs)
        m8, v8 = decode(mq, ms), r0 * r0
        m8, v8, r8 = OT.moments(g, m8, v8, self.hp, self.t)
        self.m, self.v, r = OT.moments(g, self.m, self.v, self.hp, self.t)
        self.u = ss * (self.m / (r / bc2s + eps))
        self.u8 = ss * (m8 / (r8 / bc2s + eps))
        self.w -= self.u
        self.w8 -= self.u8
        blank = (g == 0) & self.fade
        self.q = held_m(m8, blank) + encode(r8, 255)[:2]

    def roots(self):
        """The held roots over fp32's."""
        return decode(*self.q[2:]) / np.sqrt(self.v)

    def off(self):
        """What the update is off by, in its norms."""
        return np.linalg.norm(self.u8 - self.u) / np.linalg.norm(self.u)


class Noise:
    def __init__(self, spread=0.0, seed=0):
        self.rng = np.random.default_rng(seed)
        self.sigma = 1e-3 * np.exp(spread *
                                   self.rng.standard_normal((NB, BLOCK)))

    def __call__(self):
        x = self.rng.standard_normal((NB, BLOCK)) + 0.1
        return (x * self.sigma).astype(F)


def rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


def test_rules_are_the_oracles():
    rng = np.random.default_rng(1)
    m = (rng.standard_normal((NB, BLOCK)) *
         np.exp(3 * rng.standard_normal((NB, BLOCK)))).astype(F)
    m[3] = 0
    m[4] *= F(2.0 ** -120)
    blank = rng.random((NB, BLOCK)) < 0.5
    blank[5], blank[6] = True, False
    for top, x in ((127, m), (255, np.abs(m))):
        q, S, _ = encode(x, top)
        k, T = OT.encode(x.reshape(-1), top)
        assert np.array_equal(q.reshape(-1), k) and np.array_equal(S[:, 0], T)
    k, T = OT.encode(m.reshape(-1), 127)
    k = OT.faded(k, m.reshape(-1), blank.reshape(-1))
    q, S = held_m(m, blank)
    assert np.array_equal(q.reshape(-1), k) and np.array_equal(S[:, 0], T)
    assert (q != encode(m, 127)[0]).any()


# ---- elements without gradients

@pytest.mark.parametrize("spread,rate", [(0.0, (0.2, 0.5)),
                                         (1.0, (0.02, 0.2))])
def test_weights_without_gradients_come_to_rest(spread, rate):
    """An eighth of each block has no gradient after step 300.  What is left of
    m moves their weights by some lr, as in fp32; held to the nearest code
    alone they would, once their codes are small, move on by `rate` lr a
    step."""
    dead = np.zeros((NB, BLOCK), bool)
    dead[:, ::8] = True
    for fade in (True, False):
        new, T = Noise(spread), Training(fade=fade)
        for t in range(1500):
            T.step(np.where(dead & (t >= 300), F(0), new()))
            if t in (299, 899):
                at = (T.w8[dead], T.w[dead]) if t == 299 else at + (
                    T.w8[dead],)
        w8, w, later = at
        left = rms(T.w[dead] - w)
        assert 2 < left < 4
        if fade:
            assert rms((T.w8[dead] - w8) - (T.w[dead] - w)) < left / 3
            assert np.array_equal(T.w8[dead], later)
            assert not T.q[0][dead].any()
        else:
            assert rate[0] < rms(T.u8[dead]) < rate[1]


@pytest.mark.parametrize("share", [0.5, 0.9, 0.99])
def test_sporadic_gradients_move_weights_as_far(share):
    """Elements that have a gradient in few steps only: the codes that are
    rounded towards zero are too small to matter."""
    new, T = Noise(), Training()
    rng = np.random.default_rng(2)
    for t in range(2000):
        T.step(np.where(rng.random((NB, BLOCK)) < share, F(0), new()))
        if t == 499:
            a, b = T.w8.copy(), T.w.copy()
    d8, d = T.w8 - a, T.w - b
    assert abs(d8.mean() / d.mean() - 1) < 0.02
    assert rms(d8 - d) < 0.06 * rms(d)


def test_a_whole_block_without_gradients_is_fp32s():
    """Codes stay and scales fade: the moves are level with fp32's."""
    new, T = Noise(), Training()
    for t in range(1500):
        g = new()
        if t >= 300:
            g[:4] = 0
        if t == 300:
            a, b = T.w8.copy(), T.w.copy()
        T.step(g)
    d8, d = (T.w8 - a)[:4], (T.w - b)[:4]
    assert rms(d8 - d) < 0.05 * rms(d) and rms(d) < 10


@pytest.mark.parametrize("fall,like_fp32", [(1e-1, True), (1e-2, True),
                                            (1e-3, True), (1e-6, False)])
def test_gradients_that_fall(fall, like_fp32):
    """Half a block's gradients fall: down to a thousandth the weights go as
    far as in fp32, far below they move by codes of 1, about a quarter of lr a
    step to one side."""
    low = np.zeros((NB, BLOCK), bool)
    low[:, ::2] = True
    new, T = Noise(), Training()
    for t in range(2500):
        g = new()
        T.step(np.where(low, g * F(fall), g) if t >= 500 else g)
        if t == 1499:
            a, b = T.w8[low], T.w[low]
    move8, move = rms(T.w8[low] - a) / 1000, rms(T.w[low] - b) / 1000
    if like_fp32:
        assert abs(move8 / move - 1) < 0.1
    else:
        assert 0.15 < move8 < 0.5 and move < 0.12


# ---- the roots of v

@pytest.mark.parametrize("beta2,stays", [(0.95, 39), (0.98, 99), (0.99, 199),
                                         (0.995, 255), (0.999, 255)])
def test_codes_of_roots_that_stay(beta2, stays):
    """A root that a step without a gradient takes sqrt(beta2) of keeps its
    code up to a half step of it, beside an A that stays."""
    q = np.arange(1, 256)
    r = OT.decode(q, F([1 / 255 ** 2]))
    down = np.where(q == 255, r, r * F(beta2) ** F(0.5)).astype(F)
    k = OT.encode(down, 255)[0]
    assert np.array_equal(k == q, (q <= stays) | (q == 255))
    assert np.all(k[(q > stays) & (q < 255)] < q[(q > stays) & (q < 255)])


@pytest.mark.parametrize("beta2,spread,steps,root,off", [
    (0.95, 0.0, 3000, (0.99, 1.01), (0.005, 0.03)),
    (0.95, 0.3, 3000, (0.99, 1.01), (0.01, 0.04)),
    (0.95, 1.0, 3000, (0.98, 1.02), (0.03, 0.12)),
    (0.98, 0.0, 3000, (0.99, 1.01), (0.005, 0.03)),
    (0.99, 0.0, 3000, (0.98, 1.02), (0.005, 0.04)),
    (0.995, 0.0, 3000, (0.98, 1.04), (0.01, 0.05)),
    (0.999, 0.3, 4000, (0.97, 1.04), (0.02, 0.08)),
    (0.999, 1.0, 4000, (0.97, 1.04), (0.05, 0.15)),
    (0.999, 0.0, 4000, (1.08, 1.30), (0.08, 0.25)),
    (0.999, 0.0, 16000, (1.25, 1.60), (0.20, 0.40))])
def test_updates_after_many_steps(beta2, spread, steps, root, off):
    """The held roots over fp32's, and what an update is off by."""
    new, T = Noise(spread), Training(beta2=beta2)
    for _ in range(steps):
        T.step(new())
    assert root[0] < T.roots().mean() < root[1]
    assert off[0] < T.off() < off[1]


@pytest.mark.parametrize("beta2,root", [(0.95, (0.98, 1.05)),
                                        (0.99, (0.98, 1.10)),
                                        (0.999, (5.0, 12.0))])
def test_roots_of_gradients_that_fall_to_a_tenth(beta2, root):
    """Half a block's, 5000 steps later."""
    low = np.zeros((NB, BLOCK), bool)
    low[:, ::2] = True
    new, T = Noise(), Training(beta2=beta2)
    for t in range(6000):
        g = new()
        T.step(np.where(low, g * F(0.1), g) if t >= 1000 else g)
    assert root[0] < T.roots()[low].mean() < root[1]
