"""The 64-bit references of the routing and expert operators, pinned on their
own: gradients against central differences, formats against torch's casts and
closed forms, selection against a plain sort, the balance loss at its minimum."""
import numpy as np
import pytest

import operator_refs as ref


@pytest.mark.parametrize("sigmoid,renorm,K,E", [(False, False, 3, 7), (False, True, 2, 5),
                                                (True, False, 1, 4), (True, True, 4, 6),
                                                (False, True, 4, 4)])
def test_route_gradient_against_differences(sigmoid, renorm, K, E):
    rng = np.random.default_rng(K * 100 + E)
    x = rng.standard_normal((5, E))
    dw, dl, coef, scale = rng.standard_normal((5, K)), 1.7, 0.3, 2.5
    ids = ref.route(x, K, sigmoid, renorm, scale)["ids"]

    def f(x):
        o = ref.route(x, K, sigmoid, renorm, scale, None, coef, ids)
        return (o["weights"] * dw).sum() + dl * o["loss"]

    d, _ = ref.route_grad(x, ids, dw, dl, sigmoid, renorm, scale, coef)
    h = 1e-5
    for t in range(5):
        for e in range(E):
            up, dn = x.copy(), x.copy()
            up[t, e] += h
            dn[t, e] -= h
            assert abs((f(up) - f(dn)) / (2 * h) - d[t, e]) < 1e-8


def test_balance_loss_is_its_coefficient_when_balanced():
    """Equal probabilities everywhere: E/(K n^2) * sum C * n/E = 1 for any C."""
    o = ref.route(np.zeros((12, 6)), 2, coef=0.25)
    assert abs(o["loss"] - 0.25) < 1e-15
    assert (o["ids"] == [0, 1]).all()  # ties: the lower ids first


def test_masked_rows():
    x = np.array([[-np.inf, 1.0, -np.inf, 0.0], [-np.inf] * 4])
    for sg in (False, True):
        o = ref.route(x, 3, sigmoid=sg, renorm=True)
        assert o["ids"].tolist() == [[1, 3, 0], [0, 1, 2]]
        assert o["weights"][0, 2] == 0 and (o["weights"][1] == 0).all()


def test_e2m1_and_e4m3_values():
    import torch
    b = torch.arange(127, dtype=torch.uint8)
    assert (ref.E4M3 == b.view(torch.float8_e4m3fn).double().numpy()).all()
    # nearest even over a dense range, against torch's cast
    v = np.linspace(-448, 448, 100001).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    got = np.sign(v) * ref.E4M3[ref._to_grid(np.abs(v.astype(np.float64)), ref.E4M3)]
    assert (got == want).all()
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    assert ref.E2M1[ref._to_grid(ties, ref.E2M1)].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]


def test_scales():
    x = np.zeros((5, 32))
    x[1, 3], x[2, 0], x[3, 31], x[4, 5] = 6.0, 7.9, -449.0, np.inf
    x[3, 1] = 448.0
    assert ref.mx_scale(x, 4)[:, 0].tolist() == [0, 127, 127, 133, 255]
    assert ref.mx_scale(x, 8)[:, 0].tolist() == [0, 121, 122, 128, 255]
    q, s = ref.mx4(x)
    v = ref.mx4_values(q, s)
    assert v[1, 3] == 6.0 and v[2, 0] == 6.0 and v[3, 31] == -384.0 and np.isnan(v[4]).all()
    c = ref.mx_codes(x, ref.mx_scale(x, 8), 8)
    assert ref.mx_values(c, ref.mx_scale(x, 8), 8)[3, 31] == -448.0


def test_no_8_bit_value_saturates():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((400, 32)) * np.exp2(rng.integers(-20, 20, (400, 1)))
    s = ref.mx_scale(x, 8)
    v = ref.mx_values(ref.mx_codes(x, s, 8), s, 8)
    big = np.abs(x) >= np.abs(x).max(1, keepdims=True) * 2.0 ** -6
    assert (np.abs(v - x) <= 2.0 ** -4 * np.abs(x))[big].all()


def test_silu_slope_against_differences():
    g = np.linspace(-20, 20, 401)
    h = 1e-5
    assert np.abs((ref.silu(g + h) - ref.silu(g - h)) / (2 * h) - ref.silu_slope(g)).max() < 1e-9
