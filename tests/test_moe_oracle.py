"""Pins of the fp64 oracle of the norm, the routing and the experts' products: closed forms and
brute force on tiny inputs."""
import itertools
import math

import numpy as np

from oracle import moe_oracle as O


def test_norm_closed_forms():
    x = np.array([[3.0, 4.0, 0.0, 0.0], [0.0, 0.0, 0.0, 0.0]])
    r, y = O.rms_norm(x, None, np.ones(4), 0.25)
    assert np.allclose(y[0], x[0] / math.sqrt(25 / 4 + 0.25)) and np.all(y[1] == 0) and np.all(r == x)
    rng = np.random.default_rng(1)
    a, b, w = rng.standard_normal((5, 33)), rng.standard_normal((5, 33)), rng.standard_normal(33)
    r, y = O.rms_norm(a, b, w, 0.0)
    assert np.allclose(r, a + b)
    assert np.allclose(((y / w) ** 2).mean(1), 1.0)                       # unit mean square
    assert np.allclose(O.rms_norm(7 * a, 7 * b, w, 0.0)[1], y)            # scale invariance


def test_group_scales():
    y = np.zeros((1, 300))
    y[0, 5], y[0, 290] = -896.0, 4.48
    assert np.allclose(O.group_scales(y), [[2.0, 1.0, 0.01]])


def test_scores():
    l = np.array([-3.0, 0.0, 2.0])
    assert np.allclose(O.score("sigmoid", l), 1 / (1 + np.exp(-l)))
    assert np.allclose(O.score("sqrt_softplus", l) ** 2, np.log(1 + np.exp(l)))
    assert np.isclose(O.score("softmax", l).sum(), 1) and np.allclose(np.diff(np.log(O.score("softmax", l))), np.diff(l))
    for fn in ("softmax", "sigmoid", "sqrt_softplus"):
        assert np.all(O.score(fn, np.full(3, -np.inf)) == 0)


def test_route_is_the_best_set_by_brute_force():
    rng = np.random.default_rng(2)
    l, b = rng.standard_normal((40, 8)), 0.3 * rng.standard_normal(8)
    ids, w = O.route(l, b, fn="sigmoid", topk=2, n_group=4, topk_group=2, renorm=True, routed_scale=2.5)
    c = 1 / (1 + np.exp(-l)) + b
    for t in range(40):
        pair = c[t].reshape(4, 2).sum(1)
        groups = max(itertools.combinations(range(4), 2), key=lambda g: pair[list(g)].sum())
        cand = [e for e in range(8) if e // 2 in groups]
        best = max(itertools.permutations(cand, 2), key=lambda p: (c[t, p[0]], c[t, p[1]]))
        assert tuple(ids[t]) == best
        s = (c[t] - b)[list(best)]
        assert np.allclose(w[t], 2.5 * s / s.sum())


def test_route_ties_go_to_the_lower_index():
    ids, w = O.route(np.zeros((1, 6)), None, fn="softmax", topk=3, n_group=3, topk_group=2, renorm=False)
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(w, 1 / 6)


def test_expert_mlp_closed_forms():
    rng = np.random.default_rng(3)
    x, w13, w2 = rng.standard_normal((3, 4)), rng.standard_normal((2, 6, 4)), rng.standard_normal((2, 4, 3))
    ids, wt = np.array([[0, 1], [1, 1], [-1, 2]]), np.array([[0.5, 2.0], [1.0, 3.0], [9.0, 9.0]])
    out = O.expert_mlp(x, ids, wt, w13, w2)
    one = [[w2[e] @ ((g := w13[e, :3] @ x[t]) / (1 + np.exp(-g)) * (w13[e, 3:] @ x[t])) for e in range(2)] for t in range(3)]
    assert np.allclose(out[0], 0.5 * one[0][0] + 2 * one[0][1])
    assert np.allclose(out[1], 4 * one[1][1])          # named twice: counted twice
    assert np.all(out[2] == 0)                          # dropped
    lim = O.expert_mlp(x, ids, wt, 1e6 * np.abs(w13), w2, limit=2.0)   # every product of x > 0 clamps
    lim_pos = O.expert_mlp(np.abs(x), ids, wt, 1e6 * np.abs(w13), w2, limit=2.0)
    h = 2 / (1 + math.exp(-2)) * 2
    assert np.allclose(lim_pos[0], h * (0.5 * w2[0].sum(1) + 2 * w2[1].sum(1))) and np.isfinite(lim).all()
