"""The 64-bit restatements that the GPU tests compare with, checked on their own: gradients
against central differences, and a few values worked out by hand."""
import numpy as np
import pytest

import moe_reference as ref


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_is_the_difference_quotient(score, renorm):
    rng = np.random.default_rng(1)
    x = rng.standard_normal(9)
    x[4] = ref.NEG
    chosen = [7, 2, 0, -1]
    dw, ds = rng.standard_normal(4), rng.standard_normal(9)

    def loss(v):
        return (ref.route_weights(v, chosen, score, renorm, 2.5) * dw).sum() + \
            (ref.route_scores(v, score) * ds)[v > ref.NEG].sum()

    got = ref.route_backward_token(x, chosen, dw, ds, score, renorm, 2.5)
    h = 1e-5
    for e in range(9):
        if e == 4:
            assert got[e] == 0.0
            continue
        a, b = x.copy(), x.copy()
        a[e] += h
        b[e] -= h
        # central differences: error O(h^2) = 1e-10 and rounding 1e-16 / h = 1e-11
        assert abs((loss(a) - loss(b)) / (2 * h) - got[e]) < 1e-8


@pytest.mark.parametrize("name", ["relu", "gelu", "silu", "swiglu", "geglu", "none"])
def test_activation_gradient_is_the_difference_quotient(name):
    rng = np.random.default_rng(2)
    z = rng.standard_normal((3, 8)) * 2
    dy = rng.standard_normal((3, 4 if name in ("swiglu", "geglu") else 8))
    got = ref.act_backward(name, dy, z)
    h = 1e-5
    for i in np.ndindex(*z.shape):
        a, b = z.copy(), z.copy()
        a[i] += h
        b[i] -= h
        d = ((ref.act(name, a) - ref.act(name, b)) * dy).sum() / (2 * h)
        assert abs(d - got[i]) < 1e-8


def test_route_by_hand():
    # ties go to the lower index; the mask leaves two of the three slots
    assert ref.route_token([1.0, 3.0, 3.0, 1.0], 3)[0] == [1, 2, 0]
    e, w, _ = ref.route_token([0.0, ref.NEG, 0.0], 3)
    assert e == [0, 2, -1] and np.allclose(w, [0.5, 0.5, 0.0])
    # the second group's best two (0.9 + 0.8 as logits) beat the first's single best
    e, _, _ = ref.route_token([2.0, -9.0, 1.5, 1.4], 2, bias=[0, 0, 0, 0], score="sigmoid",
                              groups=2, top_groups=1, group_best=2)
    assert e == [2, 3]
    # a bias moves the choice, not the weight
    e, w, _ = ref.route_token([0.0, 0.0], 1, bias=[0.0, 1.0], score="sigmoid", renorm=False)
    assert e == [1] and w[0] == 0.5


def test_dispatch_by_hand():
    off, row_index, row_of = ref.dispatch([[1, 0], [1, -1], [0, 1]], 3)
    assert off.tolist() == [0, 2, 5, 5]
    assert row_index.tolist() == [0, 2, 0, 1, 2, -1]
    assert row_of.tolist() == [[2, 0], [3, -1], [1, 4]]
    big = np.random.default_rng(0).integers(-1, 7, (2000, 2))
    flat = big.reshape(-1)
    off, row_index, row_of = ref.dispatch(big, 7)
    for r in (0, 17, off[-1] - 1):
        p = np.nonzero(row_of.reshape(-1) == r)[0][0]
        e = flat[p]
        assert row_index[r] == p // 2 and off[e] <= r < off[e + 1]
        assert r - off[e] == (flat[:p] == e).sum()
