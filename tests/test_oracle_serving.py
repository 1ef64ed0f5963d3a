"""The serving oracle's own pins (CPU): the codes' values, the scale rule, exactness in bf16, and the
law of the tokens that the draft check gives out."""

import numpy as np
import pytest

from oracle import serving as sv


@pytest.mark.parametrize("kind,top", [(sv.FP8, 448.0), (sv.FP4, 6.0)])
def test_codes_and_scales(kind, top):
    grid = sv.GRID[kind]
    assert grid[-1] == top and len(grid) == (127 if kind == sv.FP8 else 8) and (np.diff(grid) > 0).all()
    rng = np.random.RandomState(1)
    x = (rng.randn(200, 64) * 2.0 ** rng.randint(-60, 60, (200, 1))).astype(np.float32)
    codes, scales = sv.quantise(x, kind)
    v = sv.values(codes, scales, kind)
    # nothing saturates, the scale is the smallest that holds the maximum, and errors are half a step
    amax = np.abs(x.astype(np.float64)).reshape(200, 2, 32).max(-1)
    unit = 2.0 ** (scales.astype(np.float64) - 127)
    assert (amax <= top * unit).all() and (amax > top * unit / 2).all()
    step = np.maximum(np.abs(v) / (8 if kind == sv.FP8 else 2), (2.0 ** -9 if kind == sv.FP8 else 0.5) * unit.repeat(32, 1))
    assert (np.abs(v - x) <= step).all()
    # a second pass changes nothing, and every value is exact in bf16
    assert np.array_equal(sv.held(v.astype(np.float32), kind), v)
    assert np.array_equal(sv.held(v.astype(np.float32), sv.BF16), v)


def test_ties_go_to_the_even_code():
    x = np.zeros((1, 32), np.float32)
    x[0, :9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5]
    codes, scales = sv.quantise(x, sv.FP4)
    assert scales[0, 0] == 127
    assert codes[0, :9].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 14]


def test_limits():
    for kind, high in ((sv.FP8, 119), (sv.FP4, 125)):
        x = np.zeros((4, 32), np.float32)
        x[1, 0] = np.finfo(np.float32).max
        x[2, 5] = np.inf
        x[3, 7] = 1e-40
        codes, scales = sv.quantise(x, kind)
        assert scales[:, 0].tolist() == [27, high + 127, 255, 27]
        v = sv.values(codes, scales, kind)
        assert (v[0] == 0).all() and v[1, 0] == sv.GRID[kind][-1] * 2.0 ** high and np.isnan(v[2]).all() and (v[3] == 0).all()
        assert np.isfinite(np.float32(v[1, 0]))


def test_drafts_keep_the_targets_law():
    # over many trials the first token out has the target's law whatever the draft's: the counts stay within
    # five standard deviations of it
    rng = np.random.RandomState(3)
    p, q = np.array([0.5, 0.2, 0.2, 0.1, 0.0]), np.array([0.1, 0.5, 0.1, 0.1, 0.2])
    n = 20000
    tokens = rng.choice(5, (n, 1), p=q)
    target = np.broadcast_to(p, (n, 2, 5))
    draft = np.broadcast_to(q, (n, 1, 5))
    accepted, out = sv.verify(target, draft, tokens, None, rng.rand(n, 1), rng.exponential(size=(n, 5)))
    got = np.bincount(out[:, 0], minlength=5)
    assert (np.abs(got - n * p) <= 5 * np.sqrt(n * p * (1 - p)) + 1e-9).all()
    # accepted with probability sum min(p, q)
    rate = np.minimum(p, q).sum()
    assert abs(accepted.mean() - rate) <= 5 * np.sqrt(rate * (1 - rate) / n)


def test_draw_edges():
    e = np.array([1.0, 0.5, 0.5, 2.0], np.float32)
    assert sv.draw(np.array([0, 1, 1, 0], np.float32), e) == 1          # equals: the lowest index
    assert sv.draw(np.array([0, 0, 0, 0], np.float32), e) == -1
    assert sv.draw(np.array([np.nan, 0, 0, 1], np.float32), e) == 3
    assert sv.draw(np.array([1, 0, 0, 1], np.float32), np.array([0, 1, 1, 1], np.float32)) == 0
