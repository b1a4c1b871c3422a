"""The oracle of the RMS norm with the residual's addition: its gradients
against central differences, and its scales on rows written out."""
import numpy as np
import pytest

from oracle import rmsnorm as orn


def test_gradients_against_differences():
    g = np.random.default_rng(1)
    x, r, w = g.standard_normal((3, 7)), g.standard_normal((3, 7)), g.standard_normal(7)
    dy, dh = g.standard_normal((3, 7)), g.standard_normal((3, 7))
    _, h = orn.oracle_fwd(x, r, w)
    got = orn.oracle_bwd(h, w, dy, dh)

    def loss(x, r, w):
        y, h = orn.oracle_fwd(x, r, w)
        return (y * dy).sum() + (h * dh).sum()

    for i, want in ((0, got["d"]), (1, got["d"]), (2, got["dweight"])):
        for at in np.ndindex(want.shape):
            args = [[a.copy() for a in (x, r, w)] for _ in range(2)]
            args[0][i][at] += 1e-5
            args[1][i][at] -= 1e-5
            assert abs((loss(*args[0]) - loss(*args[1])) / 2e-5 - want[at]) < 1e-8


@pytest.mark.parametrize("block,want", [(None, [[3.0 / 448], [1.0]]), (2, [[2.0 / 448, 3.0 / 448], [1.0, 1.0]])])
def test_scales(block, want):
    scales, each = orn.oracle_scales(np.array([[1.0, -2.0, 3.0], [0.0, 0.0, 0.0]]), block)
    assert (scales == np.array(want)).all() and each.shape == (2, 3)
