"""GPU parity of the gated activation with 8-bit saved inputs and its gradient.

The saved bytes are compared bit for bit.  A sigmoid is off by about 8 units
of 2^-24, so h by 16 of them (and 2^-8 for bf16); the gradient's terms d u s
(1 + g (1 - s)) and d g s by 32 of the terms' magnitudes, the weight's
gradient, a sum of F terms, by (F + 32) of the sum of magnitudes.  A sigmoid
below 2^-126 is 0 on the GPU (its reciprocal and exponential hold no
subnormals), so whatever it is multiplied by adds 2^-126 times its magnitude:
|c g u| to h, |c d u| (1 + |g|) and |c d g| to the gradient."""
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


def say(*a):
    print(*a, flush=True)


def step(env, plan, x, dh, w, F):
    moon, torch, dev = env
    rows = x.shape[0]
    o = dict(h=torch.full((rows, F), 77.0, dtype=torch.bfloat16, device=dev),
             saved=torch.full((rows, 2 * F), 0xEE, dtype=torch.uint8, device=dev),
             scales=torch.full((rows, F // 16), 0xEE, dtype=torch.uint8, device=dev),
             dx=torch.full((rows, 2 * F), 77.0, dtype=torch.bfloat16, device=dev),
             dw=torch.full((rows,), 77.0, device=dev))
    moon.moon_swiglu_save8(plan, x, o["h"], o["saved"], o["scales"], row_weights=w)
    moon.moon_swiglu_grad8(plan, dh, o["saved"], o["scales"], o["dx"], row_weights=w,
                           d_row_weights=o["dw"])
    torch.cuda.synchronize()
    return o


def check(env, sizes, E, P, F, weighted, seed, spread=0, behind=3):
    moon, torch, dev = env
    arrays, NvS = ref.plan_arrays(sizes, E, P)
    NvS += behind
    rng = np.random.default_rng(seed)
    rows = len(sizes) * NvS
    kind = ref.row_kinds(arrays, NvS)
    x = rng.standard_normal((rows, 2 * F)) * np.exp2(rng.integers(-spread, spread + 1, (rows, F // 16)).repeat(32, 1))
    x = torch.from_numpy(x).bfloat16()
    dh = torch.from_numpy(rng.standard_normal((rows, F))).bfloat16()
    w = torch.from_numpy(rng.standard_normal(rows).astype(np.float32))
    x[kind != 1], dh[kind != 1], w[kind != 1] = float("nan"), float("nan"), float("nan")
    plan = {k: torch.from_numpy(v).to(dev) for k, v in arrays.items()}
    o = {k: v.cpu() for k, v in step(env, plan, x.to(dev), dh.to(dev), w.to(dev) if weighted else None, F).items()}
    live = kind == 1
    xv, d = x.double().numpy()[live], dh.double().numpy()[live]
    c = w.double().numpy()[live][:, None] if weighted else np.ones((live.sum(), 1))
    s = ref.mx_scale(xv, 8)
    codes = ref.mx_codes(xv, s, 8)
    assert (o["scales"].numpy()[live] == s).all()
    assert (o["saved"].numpy()[live] == codes).all()
    h = c * ref.silu(xv[:, :F]) * xv[:, F:]
    got = o["h"].double().numpy()
    assert (np.abs(got[live] - h) <= (2.0 ** -8 + 16 * EPS) * np.abs(h) + 1e-37 +
            2.0 ** -126 * np.abs(c * xv[:, :F] * xv[:, F:])).all()
    v = ref.mx_values(codes, s, 8)
    g, u = v[:, :F], v[:, F:]
    sg = 1 / (1 + np.exp(-g))
    want = np.concatenate([c * d * u * ref.silu_slope(g), c * d * ref.silu(g)], 1)
    terms = np.concatenate([np.abs(c * d * u) * sg * (1 + np.abs(g)), np.abs(c * d * g) * sg], 1)
    tiny = 2.0 ** -126 * np.concatenate([np.abs(c * d * u) * (1 + np.abs(g)), np.abs(c * d * g)], 1)
    got = o["dx"].double().numpy()
    assert (np.abs(got[live] - want) <= 2.0 ** -8 * np.abs(want) + 32 * EPS * terms + tiny + 1e-37).all()
    t = d * ref.silu(g) * u
    dw = o["dw"].double().numpy()
    assert (np.abs(dw[live] - t.sum(1)) <= (F + 32) * EPS * np.abs(t).sum(1) + 1e-37).all()
    for k, zero, kept in (("h", 0, 77), ("dx", 0, 77), ("dw", 0, 77)):
        a = o[k].double().numpy()
        assert (a[kind == 2] == zero).all() and (a[kind == 0] == kept).all()
    assert (o["saved"].numpy()[kind != 1] == 0xEE).all()
    return plan, x.to(dev), dh.to(dev), w.to(dev)


CASES = [
    ("one row", [[1, 0]], 1, 1, 32),
    ("ragged", [[3, 0, 0, 0, 9, 0], [0, 0, 1, 16, 0, 0]], 4, 8, 96),
    ("padded", [[1, 0, 129, 0], [0, 64, 0, 127]], 2, 128, 224),
    ("wide", [[5, 2, 0]], 2, 4, 2048),
    ("odd width", [[0, 70, 0, 65]], 3, 1, 1056),
    ("many", [[5000, 300, 40]], 2, 16, 64),
    ("widest", [[2, 0]], 1, 1, 65536),
]


@pytest.mark.parametrize("label,sizes,E,P,F", CASES)
@pytest.mark.parametrize("weighted", [False, True])
def test_swiglu8(env, label, sizes, E, P, F, weighted):
    say(f"[case] swiglu8 {label} F={F} weighted={weighted}")
    check(env, sizes, E, P, F, weighted, seed=F)


def test_swiglu8_spread(env):
    """Blocks from 2^-30 to 2^6: tiny gates, saturated sigmoids."""
    say("[case] swiglu8 spread")
    check(env, [[64, 40, 0]], 2, 1, 128, True, seed=1, spread=6)


def test_non_finite_blocks(env):
    """An infinity or a NaN poisons its own block of the gradient, no other,
    and h only at its own place."""
    moon, torch, dev = env
    arrays, NvS = ref.plan_arrays([[4, 0]], 1, 1)
    plan = {k: torch.from_numpy(v).to(dev) for k, v in arrays.items()}
    x = torch.randn((NvS, 128), device=dev).bfloat16()
    x[1, 5], x[2, 64 + 40] = float("nan"), float("inf")
    o = step(env, plan, x, torch.ones((NvS, 64), dtype=torch.bfloat16, device=dev), None, 64)
    bad_h = torch.zeros((NvS, 64), dtype=torch.bool)
    bad_h[1, 5], bad_h[2, 40] = True, True
    assert torch.equal(~torch.isfinite(o["h"].cpu()), bad_h)
    bad = torch.zeros((NvS, 128), dtype=torch.bool)
    bad[1, :32], bad[1, 64:96], bad[2, 32:64] = True, True, True
    got = torch.isnan(o["dx"].cpu())
    # the up half of the gradient needs the gate only, the gate half both
    assert torch.equal(got, bad)
    assert torch.isnan(o["dw"].cpu()).tolist() == [False, True, True, False]


def test_gradient_against_differences(env):
    """Values on the 8-bit grid are kept exactly, so the gradient is that of
    the activation itself: central differences of the 64-bit value.  They are
    off by h^2 times a third derivative (1e-8), the gradient by bf16."""
    moon, torch, dev = env
    arrays, NvS = ref.plan_arrays([[2, 0]], 1, 1)
    plan = {k: torch.from_numpy(v).to(dev) for k, v in arrays.items()}
    rng = np.random.default_rng(2)
    x = ref.E4M3[rng.integers(56, 72, (NvS, 64))] * rng.choice([-1, 1], (NvS, 64))
    dh = rng.standard_normal((NvS, 32)).astype(np.float32)
    w = rng.standard_normal(NvS).astype(np.float32)
    t = lambda a, d=None: torch.from_numpy(a).to(dev).to(d or torch.float32)  # noqa: E731
    dhb = t(dh, torch.bfloat16)
    o = step(env, plan, t(x, torch.bfloat16), dhb, t(w), 32)
    d64 = dhb.double().cpu().numpy()

    def f(x, w):
        return (d64 * w[:, None] * ref.silu(x[:, :32]) * x[:, 32:]).sum()

    dx, dw = o["dx"].double().cpu().numpy(), o["dw"].double().cpu().numpy()
    for r in range(NvS):
        for k in range(64):
            up, dn = x.copy(), x.copy()
            up[r, k] += 1e-4
            dn[r, k] -= 1e-4
            diff = (f(up, w.astype(float)) - f(dn, w.astype(float))) / 2e-4
            assert abs(diff - dx[r, k]) <= 2.0 ** -8 * abs(diff) + 1e-5
        up, dn = w.astype(float), w.astype(float)
        up[r] += 1e-4
        dn[r] -= 1e-4
        assert abs((f(x, up) - f(x, dn)) / 2e-4 - dw[r]) < 1e-4


def test_rows_beyond_32_bit_offsets(env):
    """Gate and up of 2.6e9 values (5.2 GB): the last rows are their own
    activation and gradient."""
    moon, torch, dev = env
    F, rows = 4096, 320000
    arrays, NvS = ref.plan_arrays([[rows - 9, 9, 0]], 2, 1)
    plan = {k: torch.from_numpy(v).to(dev) for k, v in arrays.items()}
    g = torch.Generator(device=dev).manual_seed(4)
    x = torch.empty((NvS, 2 * F), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    dh = torch.empty((NvS, F), dtype=torch.bfloat16, device=dev).normal_(generator=g)
    o = step(env, plan, x, dh, None, F)
    for at in (slice(0, 2), slice(rows - 3, rows)):
        xv, d = x[at].double().cpu().numpy(), dh[at].double().cpu().numpy()
        h = ref.silu(xv[:, :F]) * xv[:, F:]
        assert (np.abs(o["h"][at].double().cpu().numpy() - h) <= (2.0 ** -8 + 16 * EPS) * np.abs(h) + 1e-37).all()
        s = ref.mx_scale(xv, 8)
        codes = ref.mx_codes(xv, s, 8)
        assert (o["saved"][at].cpu().numpy() == codes).all() and (o["scales"][at].cpu().numpy() == s).all()
        v = ref.mx_values(codes, s, 8)
        du = d * ref.silu(v[:, :F])
        assert (np.abs(o["dx"][at].double().cpu().numpy()[:, F:] - du) <= 2.0 ** -8 * np.abs(du) +
                32 * EPS * np.abs(d * v[:, :F]) + 1e-37).all()


def test_without_weight_gradient_failed_plan_and_graph(env):
    moon, torch, dev = env
    plan, x, dh, w = check(env, [[33, 0, 9], [0, 20, 0]], 2, 8, 160, True, seed=8)
    want = step(env, plan, x, dh, w, 160)
    dx = torch.full_like(want["dx"], 77.0)
    moon.moon_swiglu_grad8(plan, dh, want["saved"], want["scales"], dx, row_weights=w)
    assert torch.equal(dx.view(torch.int16), want["dx"].view(torch.int16))
    x2 = (x * 2).contiguous()
    want2 = step(env, plan, x2, dh, w, 160)
    buf, o = x.clone(), {k: torch.full_like(v, 77) if k != "saved" and k != "scales" else torch.full_like(v, 0xEE)
                         for k, v in want.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moon.moon_swiglu_save8(plan, buf, o["h"], o["saved"], o["scales"], row_weights=w)
        moon.moon_swiglu_grad8(plan, dh, o["saved"], o["scales"], o["dx"], row_weights=w, d_row_weights=o["dw"])
    for i in (1, 0, 1):
        buf.copy_(x2 if i else x)
        graph.replay()
        torch.cuda.synchronize()
        for k, v in (want2 if i else want).items():
            assert torch.equal(o[k].view(torch.uint8), v.view(torch.uint8)), k
        step(env, plan, x, dh, w, 160)
    side = torch.cuda.Stream(device=dev)
    h = torch.full_like(want["h"], 77)
    side.wait_stream(torch.cuda.current_stream())
    moon.moon_swiglu_save8(plan, x, h, o["saved"], o["scales"], row_weights=w, stream=side)
    side.synchronize()
    assert torch.equal(h.view(torch.int16), want["h"].view(torch.int16))
    plan["status"].fill_(4)
    o = step(env, plan, x, dh, w, 160)
    assert all((o[k].float() == v).all() for k, v in (("h", 77), ("dx", 77), ("dw", 77), ("saved", 0xEE)))


def test_refusals(env):
    moon, torch, dev = env
    arrays, NvS = ref.plan_arrays([[4, 0]], 1, 1)
    plan = {k: torch.from_numpy(v).to(dev) for k, v in arrays.items()}
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device=dev)  # noqa: E731
    u8 = lambda *n: torch.zeros(n, dtype=torch.uint8, device=dev)  # noqa: E731
    ok = dict(plan=plan, gate_up=bf(NvS, 64), h=bf(NvS, 32), saved=u8(NvS, 64), saved_scales=u8(NvS, 2))
    moon.moon_swiglu_save8(**ok)
    for bad in (dict(gate_up=bf(NvS, 32)), dict(h=bf(NvS, 32).float()), dict(saved=u8(NvS, 32)),
                dict(saved_scales=u8(NvS, 1)), dict(row_weights=torch.zeros(NvS + 1, device=dev)),
                dict(gate_up=bf(NvS, 64).cpu()), dict(h=bf(2 * NvS * 32))):
        with pytest.raises(ValueError):
            moon.moon_swiglu_save8(**{**ok, **bad})
    with pytest.raises(moon.MoonError):  # 48 values: no whole blocks of 32
        moon.moon_swiglu_save8(plan, bf(NvS, 96), bf(NvS, 48), u8(NvS, 96), u8(NvS, 3))
