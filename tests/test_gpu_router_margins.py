"""Group choices that fp32 sums cannot tell apart: with a large bias a key carries the rounding of the
bias's magnitude, and the worth of a group the rounding of a sum of two such keys.  The choice is that
of the 64-bit sums all the same (include/moe.h), so indices are compared exactly.

The tokens are made in pairs of groups whose true worths differ by a few fp32 steps of one logit
(1e-9 to 1e-7), far below the rounding of the keys and far above that of the 64-bit reference (1e-13).
"""

import numpy as np
import pytest

from gpu_util import np_i
from test_gpu_router import call, check

pytestmark = pytest.mark.gpu


def near_ties(T, groups, seed):
    """[T, 2 groups] logits: every group's two sigmoids sum to nearly the same number."""
    rng = np.random.default_rng(seed)
    l = np.empty((T, 2 * groups), np.float32)
    total = rng.uniform(0.7, 1.15, size=(T, 1))
    first = rng.uniform(0.2, 0.5, size=(T, groups))
    a = np.log(first / (1 - first)).astype(np.float32)
    rest = total - 1 / (1 + np.exp(-a.astype(np.float64)))
    b = np.log(rest / (1 - rest)).astype(np.float32)
    for _ in range(2):   # a few fp32 steps away
        b = np.where(rng.random(b.shape) < 0.5, np.nextafter(b, np.float32(9)), b).astype(np.float32)
    l[:, 0::2], l[:, 1::2] = a, b
    return l


def test_a_pair_of_groups_at_a_bias_of_eight():
    l = np.array([[-1.517247, 0.25438994, -2.1216793, 0.5585481]], np.float32)
    _, o = check(l, 2, score="sigmoid", groups=2, top_groups=1, group_top=2,
                 bias=np.full(4, 8, np.float32))
    assert set(o["topk_idx"][0]) == {2, 3}


@pytest.mark.parametrize("bias", [8.0, 16.0, 20.0, 32.0, 64.0])
def test_roundings_that_all_point_one_way(bias):
    """Two groups of two whose worths are equal but for about 1e-7: the first's keys lie next
    to half a step, where they round up, and their sum m1 + m2 + 2 (3 modulo 4) up again; the
    second's round down, and their sum down again.  The fp32 worths are then up to four steps of
    a key apart, the largest distance that roundings alone can make."""
    rng = np.random.default_rng(int(bias))
    u = 2.0 ** (np.floor(np.log2(bias)) - 23)
    T = 12000
    m = rng.integers(int(0.2 / u), int(0.6 / u), size=(T, 4))
    m[:, 1] += (1 - m[:, 0] - m[:, 1]) % 4                   # the sum is 1 modulo 4
    m[:, 3] = m[:, 0] + m[:, 1] - m[:, 2]
    m = m[(m[:, 3] > 0.1 / u) & (m[:, 3] < 0.65 / u)]
    s = (m + 0.5) * u + rng.uniform(-4e-8, 4e-8, size=m.shape)
    l = np.log(s / (1 - s)).astype(np.float32)
    _, o = check(l, 2, score="sigmoid", groups=2, top_groups=1, group_top=2,
                 bias=np.full(4, bias, np.float32))
    first = (o["topk_idx"][:, 0] < 2).mean()
    assert len(m) > 4000 and 0.2 < first < 0.8      # either group is the worthier


@pytest.mark.parametrize("bias", [0.0, 3.0, 8.0, 20.0, 100.0, -8.0, -100.0])
@pytest.mark.parametrize("groups,top", [(2, 1), (8, 3), (32, 4)])
def test_uniform_biases(groups, top, bias):
    l = near_ties(1500, groups, groups)
    for score in ("sigmoid", "softmax"):
        check(l, 2, score=score, groups=groups, top_groups=top, group_top=2,
              bias=np.full(2 * groups, bias, np.float32))


@pytest.mark.parametrize("group_top", [1, 2])
def test_uneven_biases_of_several_units(group_top):
    """Biases that make up for the scores' differences, on top of a large common one."""
    rng = np.random.default_rng(3)
    l = np.round(rng.normal(size=(1000, 64)) * 4).astype(np.float32) / 4
    s = 1 / (1 + np.exp(-l[0].astype(np.float64)))
    l[1::2] = l[0]
    l[1::2, 7] += 1e-6 * np.arange(500, dtype=np.float32)
    for base in (5.0, 17.0):
        check(l, 8, score="sigmoid", groups=8, top_groups=4, group_top=group_top,
              bias=(base - s).astype(np.float32))


def lane_sums(v, E):
    """fp32 sums of [T, E] as a warp forms them: a lane adds the experts lane + 32 s in ascending
    order, then the lanes are added in five rounds of pairs."""
    p = np.zeros((v.shape[0], 256), np.float32)
    p[:, :E] = v
    lanes = np.zeros((v.shape[0], 32), np.float32)
    for s in range(8):
        lanes = lanes + p[:, 32 * s:32 * s + 32]
    for o in (16, 8, 4, 2, 1):
        lanes = lanes + lanes[:, np.arange(32) ^ o]
    return lanes[:, 0]


@pytest.mark.parametrize("E", [64, 256])
def test_softmax_weights_are_normalised_by_expf(E):
    """One logit of 0, the others one x: the largest weight is 1 / z, z = 1 + (E - 1) e^x summed in
    fp32, with e^x off by at most one ulp (expf).  An exponential whose argument is scaled to base 2
    in fp32 first is off by up to three."""
    x = np.random.default_rng(E).uniform(-5.5, -2.8, 400).astype(np.float32)
    l = np.repeat(x[:, None], E, 1)
    l[np.arange(400), np.arange(400) % E] = 0
    _, _, _, _, r = call(l, 1, score="softmax", renorm=False)
    w = np_i(r["topk_w"])[:, 0]
    near = np.exp(x.astype(np.float64)).astype(np.float32)
    got = np.zeros(400, bool)
    for e in (np.nextafter(near, np.float32(0)), near, np.nextafter(near, np.float32(1))):
        v = np.repeat(e[:, None], E, 1)
        v[np.arange(400), np.arange(400) % E] = 1
        got |= w == np.float32(1) / lane_sums(v, E)
    assert got.all(), np.flatnonzero(~got)
