"""The oracles' gate gradients far from zero, against closed forms."""
import numpy as np

from oracle import block_norm, sort


def test_slope_of_saturated_gates():
    for g in (-300.0, -40.0, -18.0, 0.5, 18.0, 40.0, 300.0):
        slope = np.exp(-abs(g)) / (1 + np.exp(-abs(g))) ** 2
        one = np.ones((1, 1))
        dg = sort.combine_grad(one, np.ones((2, 1)), one, np.array([0, 1]), 1, True, np.array([g]), np.zeros((2, 1)))[2]
        assert abs(dg[0] - slope) <= 1e-15 * slope
        for gate in (np.array([g]), np.array([[g]])):
            d = block_norm.grad(one, None, one, one, gate, None, None, None, None, 1.0, 1.0)["dgate"]
            assert abs(d.item() - slope) <= 1e-15 * slope
