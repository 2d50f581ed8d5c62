"""GPU parity of the router (ids, weights, counts, balance loss) and its
gradient against the 64-bit reference.

Tolerances, in units of e = 2^-24 (half a step of fp32): an exponential of
x - max is off by |x - max| e (the subtraction) and about 4 e, so a score by
(range + 8) e; a sum of n terms adds n e; a quotient a few e.  With c = E + 2 *
range + 64 that bounds weights, probabilities and, for S tokens summed, c + S
the sums.  A gradient is off by 4 c e times the terms it adds up (the
reference gives their magnitudes); bf16 results by 2^-8 of the value more."""
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


def run(env, x, K, flags, scale, coef, bias=None, valid=None, dw=None, dl=None, bf16=False):
    """Router and gradient on the GPU; everything back as numpy."""
    moon, torch, dev = env
    R, S, E = x.shape
    t = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    lg = t(x.astype(np.float32)).to(torch.bfloat16 if bf16 else torch.float32)
    o = dict(topk=torch.full((R, S, K), -5, dtype=torch.int32, device=dev),
             weights=torch.full((R, S, K), 9.0, device=dev),
             counts=torch.full((R, E), -5, dtype=torch.int32, device=dev),
             tokens=torch.full((R,), -5, dtype=torch.int32, device=dev),
             P=torch.full((R, E), 9.0, device=dev), loss=torch.full((R,), 9.0, device=dev),
             d=torch.full((R, S, E), 9.0, dtype=lg.dtype, device=dev))
    v = t(valid)
    moon.moon_route(lg, o["topk"], o["weights"], flags, scale, bias=t(bias), valid=v,
                    tokens_per_expert=o["counts"], valid_tokens=o["tokens"], prob_sums=o["P"],
                    loss=o["loss"], loss_coef=coef)
    moon.moon_route_backward(lg, o["topk"], o["d"], flags, scale, valid=v, d_weights=t(dw),
                             tokens_per_expert=o["counts"], valid_tokens=o["tokens"],
                             d_loss=t(dl), loss_coef=coef)
    torch.cuda.synchronize()
    return {k: a.double().cpu().numpy() for k, a in o.items()}, lg.double().cpu().numpy()


def check(env, x, K, sigmoid, renorm, scale=1.0, coef=0.01, bias=None, valid=None, bf16=False,
          seed=0, loss_only=False):
    moon = env[0]
    rng = np.random.default_rng(seed)
    R, S, E = x.shape
    flags = (moon.MOON_ROUTE_SIGMOID if sigmoid else 0) | (moon.MOON_ROUTE_RENORM if renorm else 0)
    dw = None if loss_only else rng.standard_normal((R, S, K)).astype(np.float32)
    dl = (rng.standard_normal(R) * S).astype(np.float32)
    o, x = run(env, x, K, flags, scale, coef, bias, valid, dw, dl, bf16)
    b64 = None if bias is None else bias.astype(np.float64)
    for r in range(R):
        ok = np.ones(S, bool) if valid is None else valid[r].astype(bool)
        xr = x[r][ok]
        n = len(xr)
        fin = np.where(np.isfinite(xr), xr, 0.0)
        span = np.ptp(fin, axis=1).max() if n else 0.0
        c = (E + 2 * max(span, np.abs(fin).max() if n else 0.0) + 64) * EPS
        w = ref.route(xr, K, sigmoid, renorm, np.float32(scale), b64, np.float32(coef))
        ids = o["topk"][r][ok].astype(int)
        assert (ids == w["ids"]).all()
        assert (o["topk"][r][~ok] == 0).all() and (o["weights"][r][~ok] == 0).all()
        assert (np.abs(o["weights"][r][ok] - w["weights"]) <= c * w["weights"] + 1e-37).all()
        want = w["C"].copy()
        want[0] += K * (S - n)
        assert (o["counts"][r] == want).all() and o["tokens"][r] == n
        assert (np.abs(o["P"][r] - w["P"]) <= (c + S * EPS) * w["P"] + 1e-36).all()
        assert abs(o["loss"][r] - w["loss"]) <= (c + (S + E) * EPS) * abs(w["loss"]) + 1e-36
        d, terms = ref.route_grad(xr, ids, None if dw is None else dw[r][ok].astype(np.float64),
                                  float(dl[r]), sigmoid, renorm, np.float32(scale),
                                  np.float32(coef))
        got = o["d"][r]
        assert (got[~ok] == 0).all()
        assert (np.abs(got[ok] - d) <= 4 * c * terms + (2.0 ** -8 * np.abs(d) if bf16 else 0) + 1e-36).all()
    return o


@pytest.mark.parametrize("R,S,E,K,sigmoid,renorm,bf16", [
    (1, 1, 1, 1, False, True, False),        # one of everything
    (1, 1, 5, 5, True, True, False),         # every expert picked
    (2, 3, 64, 1, False, False, True),
    (3, 17, 65, 2, True, False, False),      # one expert into a second word
    (8, 16, 256, 8, True, True, True),       # a decode step
    (2, 257, 60, 6, False, False, True),     # the first size with two launches
    (4, 300, 128, 4, False, True, False),
    (2, 1000, 384, 8, False, True, False),
    (1, 500, 511, 64, True, True, False),    # the most experts per token
    (32, 33, 512, 8, False, True, True),     # the most ranks and experts
    (5, 130, 321, 7, True, False, False),
    (1, 3000, 192, 3, False, True, False),
])
def test_route(env, R, S, E, K, sigmoid, renorm, bf16):
    say(f"[case] route R={R} S={S} E={E} K={K} sigmoid={sigmoid} renorm={renorm} bf16={bf16}")
    rng = np.random.default_rng(S * 1000 + E)
    x = (2.0 * rng.standard_normal((R, S, E))).astype(np.float32)
    valid = rng.random((R, S)) < 0.7
    check(env, x, K, sigmoid, renorm, scale=2.5, bf16=bf16, seed=S)
    check(env, x, K, sigmoid, renorm, scale=2.5, bf16=bf16, seed=S, valid=valid)
    check(env, x, K, sigmoid, renorm, bf16=bf16, seed=S, valid=valid, loss_only=True)


@pytest.mark.parametrize("S", [5, 700])
def test_route_selection_bias(env, S):
    """Biased scores, many of them nearly equal: 200 distinct logits over 256
    experts with a bias that nearly undoes their scores, so the 32-bit sums tie
    where the 64-bit ones do not."""
    say(f"[case] biased routing S={S}")
    rng = np.random.default_rng(S)
    x = rng.standard_normal((2, S, 256)).astype(np.float32)
    bias = (0.05 * rng.standard_normal(256)).astype(np.float32)
    check(env, x, 8, True, True, 2.5, bias=bias)
    row = rng.standard_normal(256).astype(np.float32)
    near = np.broadcast_to(row, (2, S, 256)).copy()
    bias = (1.0 - 1.0 / (1.0 + np.exp(-row.astype(np.float64)))).astype(np.float32)
    check(env, near, 8, True, False, bias=bias)
    check(env, np.zeros((1, S, 64), np.float32), 8, True, True, bias=np.zeros(64, np.float32))


@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_ties_and_zeros(env, sigmoid):
    say(f"[case] ties sigmoid={sigmoid}")
    rng = np.random.default_rng(5)
    x = rng.integers(-2, 3, (2, 400, 200)).astype(np.float32)
    x[x == 0] = rng.choice([0.0, -0.0], (x == 0).sum())
    check(env, x, 8, sigmoid, True)
    check(env, x, 8, sigmoid, True, bf16=True)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_masked_experts(env, sigmoid, renorm):
    """-inf masks an expert; rows with fewer than K left, one left and none."""
    say(f"[case] masks sigmoid={sigmoid} renorm={renorm}")
    rng = np.random.default_rng(6)
    x = rng.standard_normal((2, 40, 70)).astype(np.float32)
    x[rng.random(x.shape) < 0.5] = -np.inf
    x[0, 3], x[0, 4, 1:], x[1, 7, :66] = -np.inf, -np.inf, -np.inf
    x[1, 8] = np.finfo(np.float32).min  # the lowest number masks nothing by itself
    check(env, x, 8, sigmoid, renorm)
    if sigmoid:
        check(env, x, 8, sigmoid, renorm, bias=rng.standard_normal(70).astype(np.float32))


def test_route_nothing_valid(env):
    """A rank whose tokens are all outside the batch, with NaN logits there."""
    x = np.random.default_rng(7).standard_normal((2, 300, 48)).astype(np.float32)
    valid = np.ones((2, 300), bool)
    valid[1], valid[0, 100:] = False, False
    x[~valid] = np.nan
    o = check(env, x, 4, False, True, valid=valid)
    assert o["loss"][1] == 0 and o["counts"][1, 0] == 1200 and o["tokens"][1] == 0


def test_route_nan_and_infinite_logits(env):
    """Ids stay distinct and in range; the token's softmax weights are NaN."""
    moon, torch, dev = env
    x = np.random.default_rng(8).standard_normal((1, 4, 100)).astype(np.float32)
    x[0, 1, 50], x[0, 2], x[0, 3, 7] = np.nan, np.nan, np.inf
    o, _ = run(env, x, 6, moon.MOON_ROUTE_RENORM, 1.0, 0.0)
    for t in range(4):
        ids = o["topk"][0, t]
        assert len(set(ids)) == 6 and ids.min() >= 0 and ids.max() < 100
    assert 50 not in o["topk"][0, 1] and o["topk"][0, 2].tolist() == [0, 1, 2, 3, 4, 5]
    assert np.isfinite(o["weights"][0, 0]).all() and np.isnan(o["weights"][0, 2]).all()
    assert o["topk"][0, 3, 0] == 7 and np.isnan(o["weights"][0, 3, 0])


def test_route_gradient_against_differences(env):
    """The GPU's gradient against central differences of the 64-bit value with
    the ids and counts held.  The differences are off by h^2 times a third
    derivative (below 1e-8 here); the gradient by 32-bit rounding (1e-6 of the
    terms, which are below 4)."""
    moon = env[0]
    rng = np.random.default_rng(9)
    x = rng.standard_normal((1, 3, 9)).astype(np.float32)
    dw, dl = rng.standard_normal((1, 3, 4)).astype(np.float32), np.array([2.0], np.float32)
    for sigmoid, renorm in [(False, False), (False, True), (True, False), (True, True)]:
        flags = (moon.MOON_ROUTE_SIGMOID if sigmoid else 0) | (moon.MOON_ROUTE_RENORM if renorm else 0)
        o, x64 = run(env, x, 4, flags, 1.0, 0.5, dw=dw, dl=dl)
        ids = o["topk"][0].astype(int)

        def f(z):
            w = ref.route(z, 4, sigmoid, renorm, 1.0, None, 0.5, ids)
            return (w["weights"] * dw[0]).sum() + dl[0] * w["loss"]

        for t in range(3):
            for e in range(9):
                up, dn = x64[0].copy(), x64[0].copy()
                up[t, e] += 1e-4
                dn[t, e] -= 1e-4
                assert abs((f(up) - f(dn)) / 2e-4 - o["d"][0, t, e]) < 5e-6


def test_route_feeds_the_planner(env):
    """The counts are what moon_plan compares with its own histogram, also
    with tokens outside the batch; a different count is refused."""
    moon, torch, dev = env
    R, S, E, K = 4, 100, 16, 4
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.randn((R, S, E), generator=g, device=dev)
    valid = torch.rand((R, S), generator=g, device=dev) < 0.8
    topk = torch.empty((R, S, K), dtype=torch.int32, device=dev)
    w = torch.empty((R, S, K), device=dev)
    tpe = torch.empty((R, E), dtype=torch.int32, device=dev)
    moon.moon_route(x, topk, w, moon.MOON_ROUTE_RENORM, valid=valid, tokens_per_expert=tpe)
    ctx = moon.moon_ctx_create(R, E, K, S, 64, 0, 8)
    plan = moon.moon_plan_create(ctx)
    try:
        moon.moon_plan(ctx, topk, tpe, plan)
        assert moon.moon_plan_status(plan) == moon.MOON_OK
        tpe[1, 2] += 1
        moon.moon_plan(ctx, topk, tpe, plan)
        assert moon.moon_plan_status(plan) == moon.MOON_ERR_HISTOGRAM
    finally:
        moon.moon_plan_destroy(plan)
        moon.moon_ctx_destroy(ctx)


def test_route_only_what_is_asked(env):
    """Without optional outputs the ids and weights are the same; each output
    alone is too; a workspace of the caller's serves two calls in a row."""
    moon, torch, dev = env
    g = torch.Generator(device=dev).manual_seed(4)
    x = torch.randn((2, 600, 96), generator=g, device=dev)
    full = {}

    def call(**kw):
        topk = torch.empty((2, 600, 5), dtype=torch.int32, device=dev)
        w = torch.empty((2, 600, 5), device=dev)
        moon.moon_route(x, topk, w, 0, 1.5, loss_coef=0.1, **kw)
        return topk, w

    full = dict(tokens_per_expert=torch.empty((2, 96), dtype=torch.int32, device=dev),
                valid_tokens=torch.empty((2,), dtype=torch.int32, device=dev),
                prob_sums=torch.empty((2, 96), device=dev), loss=torch.empty((2,), device=dev))
    n = moon.moon_route_workspace(2, 600, 96, 5)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    topk, w = call(workspace=ws, **full)
    t2, w2 = call()
    assert torch.equal(topk, t2) and torch.equal(w, w2)
    for k, v in full.items():
        one = torch.zeros_like(v)
        t3, w3 = call(workspace=ws, **{k: one})
        assert torch.equal(one, v) and torch.equal(t3, topk) and torch.equal(w3, w)
    with pytest.raises(moon.MoonError):
        call(workspace=ws[:n - 4], **full)


def test_route_streams_and_graph(env):
    """On a side stream, and captured with its gradient: every replay equals
    the eager result for the inputs then in place, bit for bit."""
    moon, torch, dev = env
    R, S, E, K = 2, 400, 128, 6
    g = torch.Generator(device=dev).manual_seed(5)
    sets = [torch.randn((R, S, E), generator=g, device=dev) for _ in range(3)]
    x = sets[0].clone()
    dw = torch.randn((R, S, K), generator=g, device=dev)
    dl = torch.ones((R,), device=dev)

    def buffers():
        return dict(topk=torch.zeros((R, S, K), dtype=torch.int32, device=dev),
                    w=torch.zeros((R, S, K), device=dev),
                    c=torch.zeros((R, E), dtype=torch.int32, device=dev),
                    n=torch.zeros((R,), dtype=torch.int32, device=dev),
                    loss=torch.zeros((R,), device=dev), d=torch.zeros((R, S, E), device=dev))

    def step(x, b, stream=None):
        moon.moon_route(x, b["topk"], b["w"], 2, 1.0, tokens_per_expert=b["c"],
                        valid_tokens=b["n"], loss=b["loss"], loss_coef=0.1, stream=stream)
        moon.moon_route_backward(x, b["topk"], b["d"], 2, 1.0, d_weights=dw,
                                 tokens_per_expert=b["c"], valid_tokens=b["n"], d_loss=dl,
                                 loss_coef=0.1, stream=stream)

    want = []
    for s in sets:
        b = buffers()
        step(s, b)
        want.append(b)
    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream())
    b = buffers()
    side.wait_stream(torch.cuda.current_stream())
    step(sets[1], b, stream=side)
    side.synchronize()
    assert all(torch.equal(b[k], want[1][k]) for k in b)
    b = buffers()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x, b)
    for i in (1, 2, 0, 1):
        x.copy_(sets[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(b[k], want[i][k]) for k in b), i
        step(sets[2], buffers())  # eager work between the replays


def test_route_refusals(env):
    moon, torch, dev = env
    x = torch.zeros((2, 4, 8), device=dev)
    topk = torch.zeros((2, 4, 2), dtype=torch.int32, device=dev)
    w = torch.zeros((2, 4, 2), device=dev)
    with pytest.raises(moon.MoonError):  # bias without sigmoid scores
        moon.moon_route(x, topk, w, bias=torch.zeros(8, device=dev))
    with pytest.raises(moon.MoonError):
        moon.moon_route(x, topk, w, flags=4)
    for bad in (dict(topk=topk.long()), dict(topk=topk[:, :3]), dict(logits=x.double()),
                dict(logits=x.cpu()), dict(logits=x.transpose(0, 1)), dict(logits=x[0]),
                dict(weights=w[:1]), dict(valid=torch.zeros((2, 4), device=dev)),
                dict(bias=torch.zeros(7, device=dev), flags=1)):
        a = dict(logits=x, topk=topk, weights=w)
        a.update(bad)
        with pytest.raises(ValueError):
            moon.moon_route(**a)
    with pytest.raises(moon.MoonError):  # the loss's gradient without its counts
        moon.moon_route_backward(x, topk, torch.zeros_like(x), d_loss=torch.zeros(2, device=dev))
    with pytest.raises(ValueError):
        moon.moon_route_backward(x, topk, torch.zeros((2, 4, 8), dtype=torch.bfloat16, device=dev))


@pytest.mark.parametrize("E,K", [(70, 8), (128, 4), (384, 8), (384, 48), (512, 64)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid", "biased"])
@pytest.mark.parametrize("bf16", [False, True])
def test_route_nan_among_numbers(env, E, K, score, bf16):
    """NaN logits, quiet and signalling, of both signs: next to a lane's largest
    number, in rows with fewer than K numbers and in rows without one.  They
    rank behind -inf, and weights over numbers alone are not touched by them
    (relative error as above: the sum's terms, twice the exponent's span, 64)."""
    moon, torch, dev = env
    say(f"[case] NaN E={E} K={K} {score} bf16={bf16}")
    rng = np.random.default_rng(E + K)
    S = 60
    bits = (3.0 * rng.standard_normal((1, S, E))).astype(np.float32).view(np.uint32) & 0xFFFF0000
    nans = np.array([0x7F810000, 0xFF810000, 0x7FC00000, 0xFFC10000], np.uint32)
    part = np.linspace(0.0, 1.0, S)[None, :, None]  # the share of NaN grows by token
    bits = np.where(rng.random(bits.shape) < part, rng.choice(nans, bits.shape), bits)
    bits = np.where(rng.random(bits.shape) < 0.1, np.uint32(0xFF800000), bits)
    bits[0, -1] = nans[0]
    bits[0, 0, :] = np.where(np.arange(E) < E // 2, np.uint32(0x42F00000), nans[1])  # 120.0
    x = bits.astype(np.uint32).view(np.float32)
    lg = torch.from_numpy(x.copy()).to(dev) if not bf16 else \
        torch.from_numpy((bits >> 16).astype(np.uint16).view(np.int16)).to(dev).view(torch.bfloat16)
    bias = (rng.integers(-8, 9, E) / 4.0).astype(np.float32) if score == "biased" else None
    topk = torch.empty((1, S, K), dtype=torch.int32, device=dev)
    w = torch.empty((1, S, K), device=dev)
    moon.moon_route(lg, topk, w, moon.MOON_ROUTE_RENORM | (moon.MOON_ROUTE_SIGMOID if score != "softmax" else 0),
                    bias=None if bias is None else torch.from_numpy(bias).to(dev))
    torch.cuda.synchronize()
    topk, w = topk.cpu().numpy()[0], w.double().cpu().numpy()[0]
    for t in range(S):
        with np.errstate(invalid="ignore"):
            z = x[0, t].astype(np.float64)
        num = ~np.isnan(z)
        top = z[num & ~np.isneginf(z)].max(initial=-np.inf)
        with np.errstate(over="ignore", invalid="ignore"):
            s = 1.0 / (1.0 + np.exp(-z)) if score != "softmax" else \
                np.exp(z - (top if np.isfinite(top) else 0.0))
        key = z if bias is None else np.where(np.isneginf(z), -np.inf, s + bias)
        ids = np.lexsort((np.arange(E), -np.where(num, key, 0.0), ~num))[:K]
        assert (topk[t] == ids).all(), t
        if num[ids].all():
            den = s[ids].sum()
            want = s[ids] / (den if den > 0 else 1.0)
            assert (np.abs(w[t] - want) <= (E + 2 * 130 + 64) * EPS * want + 1e-37).all(), t
        else:
            assert np.isnan(w[t]).all(), t


def test_route_most_tokens(env):
    """2^31 - 1 tokens, the most there can be: token counters and the cut into
    workgroups stay in range (20 GB; one expert, so ids 0 and weights 1.5)."""
    moon, torch, dev = env
    say("[case] 2^31 - 1 tokens")
    S = 2 ** 31 - 1
    x = torch.zeros((1, S, 1), dtype=torch.bfloat16, device=dev)
    topk = torch.full((1, S, 1), -1, dtype=torch.int32, device=dev)
    w = torch.zeros((1, S, 1), device=dev)
    moon.moon_route(x, topk, w, 0, 1.5)
    torch.cuda.synchronize()
    for a in range(0, S, 2 ** 28):  # in parts that torch indexes with 32 bits
        assert int(topk[0, a:a + 2 ** 28].abs().max()) == 0
        assert float(w[0, a:a + 2 ** 28].min()) == 1.5 == float(w[0, a:a + 2 ** 28].max())
    x.fill_(1.0)
    d = torch.ones_like(x)
    moon.moon_route_backward(x, topk, d, 0, 1.5, d_weights=w)
    torch.cuda.synchronize()
    for a in range(0, S, 2 ** 28):  # a softmax over one expert has no gradient
        assert float(d[0, a:a + 2 ** 28].float().abs().max()) == 0.0


@pytest.mark.parametrize("S", [7, 300])
def test_route_infinite_biases(env, S):
    """A bias of infinity forces an expert, -infinity leaves it to the last, NaN
    behind those; the scores stay what they were."""
    moon, torch, dev = env
    say(f"[case] infinite biases S={S}")
    rng = np.random.default_rng(S)
    E, K = 96, 8
    x = rng.standard_normal((1, S, E)).astype(np.float32)
    x[0, 1, :60] = -np.inf
    for forced, out, nan in [([5, 70, 3], range(20, 40), [0]), (range(0, 90, 7), [1], []),
                             ([], range(0, 90), [91, 92]), ([2], range(3, 96), [])]:
        bias = np.round(rng.standard_normal(E) * 8).astype(np.float32) / 8
        bias[list(forced)], bias[list(out)], bias[list(nan)] = np.inf, -np.inf, np.nan
        topk = torch.empty((1, S, K), dtype=torch.int32, device=dev)
        w = torch.empty((1, S, K), device=dev)
        moon.moon_route(torch.from_numpy(x).to(dev), topk, w, moon.MOON_ROUTE_SIGMOID | moon.MOON_ROUTE_RENORM,
                        bias=torch.from_numpy(bias).to(dev))
        torch.cuda.synchronize()
        z = x[0].astype(np.float64)
        s = 1.0 / (1.0 + np.exp(-z))
        key = np.where(np.isneginf(z), -np.inf, s + bias)
        order = np.lexsort((np.broadcast_to(np.arange(E), key.shape),
                            -np.where(np.isnan(key), 0.0, key), np.isnan(key)))[:, :K]
        assert (topk.cpu().numpy()[0] == order).all()
        sel = np.take_along_axis(s, order, 1)
        want = sel / np.where(sel.sum(1) > 0, sel.sum(1), 1.0)[:, None]
        # a score's exponent and reciprocal, the sum's K terms, the division
        assert (np.abs(w.double().cpu().numpy()[0] - want) <= (K + 2 * 6 + 64) * EPS * want + 1e-37).all()
