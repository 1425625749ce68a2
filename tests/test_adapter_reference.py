"""The restated adapter operators (adapter_reference.py) against difference quotients."""
import numpy as np

import adapter_reference as ref


def test_backward_is_the_gradient():
    rng = np.random.default_rng(3)
    E, R, K, N, T = 3, 4, 5, 6, 9
    off, t = [0, 2, 2, 7], np.array([4, 1, 0, 8, 3, 2, 6, 5, 7])
    x, a, b = rng.standard_normal((T, K)), rng.standard_normal((E, R, K)), rng.standard_normal((E, N, R))
    scale, base, w = rng.standard_normal(E), rng.standard_normal((T, N)), rng.standard_normal((T, N))

    def loss(x, a, b):
        return float((ref.lora(x, a, b, off, t, t, scale, base)[0] * w).sum())

    out, u = ref.lora(x, a, b, off, t, t, scale, base)
    assert np.array_equal(out[[5, 7]], base[[5, 7]]) and not u[7:].any()   # rows without an adapter
    dx, da, db = ref.lora_backward(w, x, u, a, b, off, t, t, scale, np.zeros((T, K)))
    h = 1e-6
    for v, g in ((x, dx), (a, da), (b, db)):
        for _ in range(12):
            i = tuple(rng.integers(0, n) for n in v.shape)
            at = v[i]
            v[i] = at + h
            up = loss(x, a, b)
            v[i] = at - h
            down = loss(x, a, b)
            v[i] = at
            assert abs((up - down) / (2 * h) - g[i]) <= 1e-7 * (1 + abs(g[i])), (i, g[i])
    assert not da[1].any() and not db[1].any()   # an adapter without rows


def test_norm_of_values_whose_squares_leave_fp32():
    assert np.isclose(ref.norm([np.float32([3e30]), np.float32([4e30])]), 5e30, rtol=1e-7)
    assert ref.norm([]) == 0.0
