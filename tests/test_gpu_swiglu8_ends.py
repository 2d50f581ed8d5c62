"""The 8-bit scales of the saved activation at their ends: every bf16 pattern,
saved bytes compared bit for bit, and read back through the gradient."""
import numpy as np
import pytest

import operator_refs as ref

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import combine_balanced_planning_amd as moon
    return moon, torch, torch.device("cuda", 0)


def save(env, bits):
    """moon_swiglu_save8 of rows of bf16 bits [rows, 64]: (values, saved, scales)."""
    moon, torch, dev = env
    arrays, NvS = ref.plan_arrays([[bits.shape[0], 0]], 1, 1)
    plan = {k: torch.from_numpy(v).to(dev) for k, v in arrays.items()}
    x = torch.from_numpy(bits.view(np.int16)).to(dev).view(torch.bfloat16)
    h = torch.empty((NvS, 32), dtype=torch.bfloat16, device=dev)
    saved = torch.full((NvS, 64), 0xEE, dtype=torch.uint8, device=dev)
    scales = torch.full((NvS, 2), 0xEE, dtype=torch.uint8, device=dev)
    moon.moon_swiglu_save8(plan, x, h, saved, scales)
    return plan, x.double().cpu().numpy(), saved, scales


@pytest.mark.parametrize("lift", [0, 1, 2, 5, 9, 14, 17])
def test_every_bf16_pattern(env, lift):
    """All patterns as a gate and as an up value, beside a value that many
    binades up (0: alone, so that it sets the scale): rounding, ties, the border
    of 1.75 * 2^k, subnormals, scale byte 0, infinity, NaN."""
    print(f"[case] all bf16 patterns, neighbour {lift} binades up", flush=True)
    p = np.arange(65536, dtype=np.uint16)
    up = np.minimum((p & 0x7FFF).astype(np.int64) + (lift << 7), 0x7F7F).astype(np.uint16)
    up = np.where(((p & 0x7F80) == 0x7F80) | (lift == 0), 0, up).astype(np.uint16)
    bits = np.zeros((65536, 64), np.uint16)
    bits[:, 5], bits[:, 20] = p, up
    bits[:, 32 + 30], bits[:, 32 + 9] = p[::-1], up[::-1] | 0x8000
    _, v, saved, scales = save(env, bits)
    s = ref.mx_scale(v, 8)
    assert (scales.cpu().numpy() == s).all()
    assert (saved.cpu().numpy() == ref.mx_codes(v, s, 8)).all()
    finite = s != 255
    assert s[finite].min() == max(0, lift - 8) and s[finite].max() == 247


@pytest.mark.parametrize("small", [True, False])
def test_ends_read_back(env, small):
    """Blocks under the smallest scales and under the largest, as the gate and
    as the up values: the gradient of up is dh silu(g), that of gate dh u
    silu'(g), in 64 bits from the saved values.  dh moves them to ordinary
    numbers.  Bounds: bf16's rounding, 32 units of the terms, and half a
    subnormal step of fp32 (2^-150) times dh for each product before it.  A
    magnitude of 1.9375 * 2^127 or more is nearest to 2^128 in e4m3 (its step is
    2^-3 of 2^127 there), which fp32 does not hold: it reads back as infinity,
    and its own two gradients are not finite."""
    moon, torch, dev = env
    print(f"[case] ends read back small={small}", flush=True)
    rng = np.random.default_rng(small)
    rows = 600
    # bf16 exponents: the lowest 14 binades and subnormals, or the highest 6
    e = rng.integers(0, 14, (rows, 1)) if small else rng.integers(249, 255, (rows, 1))
    far = ((np.maximum(e - rng.integers(0, 4, (rows, 32)), 0) << 7) | rng.integers(0, 128, (rows, 32)) |
           (rng.integers(0, 2, (rows, 32)) << 15)).astype(np.uint16)
    one = np.full((rows, 32), 0x3F80, np.uint16)
    for gate_far in (True, False):
        bits = np.concatenate([far, one] if gate_far else [one, far], 1)
        plan, v, saved, scales = save(env, bits)
        s = ref.mx_scale(v, 8)
        assert (scales.cpu().numpy() == s).all()
        assert (s.min() == 0) if small else (s.max() >= 246)
        v = ref.mx_values(saved.cpu().numpy(), s, 8)
        g, u = v[:, :32], v[:, 32:]
        dh = np.float64(2.0 ** (100 if small else -100))
        dx = torch.empty((rows, 64), dtype=torch.bfloat16, device=dev)
        d = torch.full((rows, 32), float(dh), dtype=torch.bfloat16, device=dev)
        moon.moon_swiglu_grad8(plan, d, saved, scales, dx)
        got = dx.double().cpu().numpy()
        lost = 2 * dh * 2.0 ** -150
        over = np.maximum(np.abs(g), np.abs(u)) >= 2.0 ** 128
        assert over.any() != small
        want = np.concatenate([dh * u * ref.silu_slope(g), dh * ref.silu(g)], 1)
        near = np.abs(got - want) <= (2.0 ** -8 + 32 * EPS) * np.abs(want) + lost
        assert near[:, :32][~over].all() and near[:, 32:][~over].all()
        assert not np.isfinite(got[:, 32:] if gate_far else got[:, :32])[over].any()
