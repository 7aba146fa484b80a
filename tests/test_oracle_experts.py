"""Pins of the experts' oracle: gradients by differences, worked examples, and the products against a loop (no GPU)."""

import numpy as np

from oracle import experts


def test_sort_worked_example():
    ids = np.array([[2, 0], [0, 5], [2, -1], [0, 2]])
    row_of, starts, counts = experts.sort(ids, 4, 4)
    assert counts.tolist() == [3, 0, 3, 0] and starts.tolist() == [0, 4, 4, 8, 8]
    assert row_of.tolist() == [[4, 0], [1, -1], [5, -1], [2, 6]]
    token, zero = experts.written(starts, counts, 9)
    assert token.tolist() == [1, 1, 1, 0, 1, 1, 1, 0, 0] and zero.tolist() == [0, 0, 0, 1, 0, 0, 0, 1, 0]


def test_combine_and_its_gradient_by_differences():
    rng = np.random.default_rng(1)
    ids = np.array([[0, 1], [1, 1], [2, -1], [0, 2]])
    row_of, starts, counts = experts.sort(ids, 3, 2)
    y, w, d = rng.standard_normal((8, 5)), rng.random((4, 2)), rng.standard_normal((4, 5))
    dy, dw = experts.combine_backward(d, y, row_of, w)
    loss = lambda y, w: float((experts.combine(y, row_of, w) * d).sum())  # noqa: E731
    for x, g in ((y, dy), (w, dw)):
        for i in np.ndindex(x.shape):
            x[i] += 1e-3
            up = loss(y, w)
            x[i] -= 2e-3
            down = loss(y, w)
            x[i] += 1e-3
            assert abs((up - down) / 2e-3 - g[i]) < 1e-9


def test_dispatch_and_its_gradient_by_differences():
    rng = np.random.default_rng(2)
    row_of, starts, counts = experts.sort(np.array([[0, 1], [1, 0], [-1, 2]]), 3, 4)
    x, d = rng.standard_normal((3, 4)), rng.standard_normal((12, 4))
    dx = experts.dispatch_backward(d, row_of)
    for i in np.ndindex(x.shape):
        x[i] += 1e-3
        up = (experts.dispatch(x, row_of, 12) * d).sum()
        x[i] -= 2e-3
        down = (experts.dispatch(x, row_of, 12) * d).sum()
        x[i] += 1e-3
        assert abs((up - down) / 2e-3 - dx[i]) < 1e-9


def test_products_and_their_gradient_by_differences():
    rng = np.random.default_rng(3)
    starts = [0, 3, 3, 7]
    a, b, d = rng.standard_normal((8, 4)), rng.standard_normal((6, 4)), rng.standard_normal((8, 2))
    out = experts.product(a, b, starts)
    for e in range(3):
        for i in range(starts[e], starts[e + 1]):
            for j in range(2):
                assert abs(out[i, j] - sum(a[i, l] * b[e * 2 + j, l] for l in range(4))) < 1e-12
    assert not out[7].any()
    d[7] = 0
    db = experts.product_grad(d.T, a.T, starts)
    for i in np.ndindex(b.shape):
        b[i] += 1e-3
        up = (experts.product(a, b, starts) * d).sum()
        b[i] -= 2e-3
        down = (experts.product(a, b, starts) * d).sum()
        b[i] += 1e-3
        assert abs((up - down) / 2e-3 - db[i]) < 1e-9
