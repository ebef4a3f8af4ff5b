"""Pins of the mixture-of-experts and adapter oracle: brute force over tokens, invariants of the row plan, and
gradients against central differences of the forward pass."""
import numpy as np
import pytest

from oracle import mlp as OM
from oracle import moe as M


def _problem(seed=0, N=7, E=5, k=2, h=6, F=4, act="swiglu"):
    r = np.random.default_rng(seed)
    wide = 2 if act == "swiglu" else 1
    return (r.standard_normal((N, h)), r.standard_normal((N, E)), 0.5 * r.standard_normal((E, h, wide * F)),
            0.5 * r.standard_normal((E, F, h)), r.standard_normal((N, h)))


def test_choice_descends_and_breaks_ties_by_index():
    l = np.array([[0.0, 2.0, 2.0, 1.0], [np.nan, -np.inf, 3.0, np.inf], [-np.inf] * 4])
    assert M.choose(l, 3).tolist() == [[1, 2, 3], [3, 2, -1], [-1, -1, -1]]
    w = M.route(l, 3, "topk")["weight"]
    assert np.allclose(w[0], np.exp([0, 0, -1]) / np.exp([0, 0, -1]).sum())
    assert w[1].tolist() == [1.0, 0.0, 0.0] and w[2].tolist() == [0.0] * 3
    s = M.route(l, 3, "softmax")["weight"]
    assert np.allclose(s[0].sum() + 1 / np.exp([0, 2, 2, 1]).sum(), 1.0)


@pytest.mark.parametrize("rest", [False, True])
def test_row_plan_is_a_stable_sort(rest):
    r = np.random.default_rng(1)
    expert = r.integers(-1, 6, (50, 1 if rest else 3)).astype(np.int32)
    off, token, slot = M.sort_rows(expert, 6, rest)
    assert off[0] == 0 and (np.diff(off) >= 0).all() and len(token) == (50 if rest else off[6])
    for e in range(6):
        got = token[off[e]:off[e + 1]]
        assert got.tolist() == [n for n in range(50) for j in range(expert.shape[1]) if expert[n, j] == e]
    for n in range(50):
        for j in range(expert.shape[1]):
            if slot[n, j] >= 0:
                assert token[slot[n, j]] == n
            else:
                assert expert[n, j] == -1 and not rest


@pytest.mark.parametrize("act", OM.ACTS)
@pytest.mark.parametrize("gate", ["softmax", "topk"])
def test_mlp_is_each_tokens_own_experts(act, gate):
    x, l, w_in, w_down, _ = _problem(2, act=act)
    f = M.moe_mlp(x, l, w_in, w_down, 2, gate, act)
    for n in range(len(x)):
        ref = sum(w * OM.mlp_unsharded(x[n:n + 1], w_in[e], w_down[e], act)[0] for e, w in zip(f["expert"][n], f["weight"][n]))
        assert np.allclose(f["y"][n], ref)


@pytest.mark.parametrize("act", OM.ACTS)
@pytest.mark.parametrize("gate", ["softmax", "topk"])
def test_gradients_against_differences(act, gate):
    x, l, w_in, w_down, dy = _problem(3, act=act)
    g = M.moe_mlp_backward(x, l, w_in, w_down, 2, gate, act, dy)
    loss = lambda: float((M.moe_mlp(x, l, w_in, w_down, 2, gate, act)["y"] * dy).sum())  # noqa: E731
    r = np.random.default_rng(4)
    for v, name in ((x, "dx"), (l, "dlogits"), (w_in, "dw_in"), (w_down, "dw_down")):
        for _ in range(6):
            at = tuple(r.integers(0, s) for s in v.shape)
            old, eps = v[at], 1e-6
            v[at] = old + eps
            hi = loss()
            v[at] = old - eps
            lo = loss()
            v[at] = old
            assert abs((hi - lo) / (2 * eps) - g[name][at]) < 1e-7 * (1 + abs(g[name][at])) + 1e-8, (name, at)


def test_segments_are_clamped():
    assert M.segments([0, 3, 2, 9], 5) == [(0, 3), (3, 3), (2, 5)]
    assert M.segments([-4, 1], 5) == [(0, 1)]


def test_adapters_are_a_low_rank_change_of_the_weight():
    r = np.random.default_rng(5)
    x, w = r.standard_normal((6, 8)), r.standard_normal((2, 8, 3))
    a, b, s = r.standard_normal((4, 8, 2)), r.standard_normal((2, 4, 2, 3)), r.standard_normal(4)
    ids = np.array([1, -1, 3, 1, 7, 0])
    y = M.lora(x, w, a, b, s, ids)
    for n, i in enumerate(ids):
        for t in range(2):
            full = w[t] + (s[i] * a[i] @ b[t, i] if 0 <= i < 4 else 0.0)
            assert np.allclose(y[t, n], x[n] @ full)
