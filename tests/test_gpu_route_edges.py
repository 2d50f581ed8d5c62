"""The router and its gradient where logits are far apart, masked or far below
zero, and around the size at which a call takes a second launch; every token is
held to the tolerance of its own logits.

In units of e = 2^-24 a score is off by its exponent's argument (at most 130: a
score beyond 88 below its largest is 0 on the GPU) and about 8 more, a sum of E
terms by E and a quotient by a few: c = E + 2 * range + 64 with the range of
the token's finite logits for a softmax, their largest magnitude for a sigmoid.
Scores below 2^-126 count as 0, which a weight sees divided by the picked
scores' sum.  A gradient is off by 4 c e times the terms it adds up."""
import numpy as np
import pytest

import operator_refs as ref

pytestmark = pytest.mark.gpu
EPS, TINY = 2.0 ** -24, 2.0 ** -126


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import combine_balanced_planning_amd as moon
    return moon, torch, torch.device("cuda", 0)


def check(env, x, K, sigmoid, renorm, scale=1.0, bias=None, valid=None, dw_scale=1.0, coef=0.01, seed=0):
    """Everything that the router and its gradient write for x [R, S, E]."""
    moon, torch, dev = env
    rng = np.random.default_rng(seed)
    R, S, E = x.shape
    dw = (dw_scale * rng.standard_normal((R, S, K))).astype(np.float32)
    dl = (rng.standard_normal(R) * S * dw_scale).astype(np.float32)
    t = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    f = lambda *s: torch.full(s, 9.0, device=dev)  # noqa: E731
    i = lambda *s: torch.full(s, -5, dtype=torch.int32, device=dev)  # noqa: E731
    topk, w, counts, tokens, P, loss, d = i(R, S, K), f(R, S, K), i(R, E), i(R), f(R, E), f(R), f(R, S, E)
    flags = (moon.MOON_ROUTE_SIGMOID if sigmoid else 0) | (moon.MOON_ROUTE_RENORM if renorm else 0)
    moon.moon_route(t(x), topk, w, flags, scale, bias=t(bias), valid=t(valid), tokens_per_expert=counts,
                    valid_tokens=tokens, prob_sums=P, loss=loss, loss_coef=coef)
    moon.moon_route_backward(t(x), topk, d, flags, scale, valid=t(valid), d_weights=t(dw),
                             tokens_per_expert=counts, valid_tokens=tokens, d_loss=t(dl), loss_coef=coef)
    torch.cuda.synchronize()
    topk, w, counts, tokens, P, loss, d = (a.cpu().double().numpy() for a in (topk, w, counts, tokens, P, loss, d))
    sc, cf = np.float32(scale), np.float32(coef)
    for r in range(R):
        ok = np.ones(S, bool) if valid is None else valid[r].astype(bool)
        xr = x[r][ok].astype(np.float64)
        n = len(xr)
        want = ref.route(xr, K, sigmoid, renorm, sc, None if bias is None else bias.astype(np.float64), cf)
        ids = topk[r][ok].astype(int)
        assert (ids == want["ids"]).all()
        assert (topk[r][~ok] == 0).all() and (w[r][~ok] == 0).all() and (d[r][~ok] == 0).all()
        load = want["C"].copy()
        load[0] += K * (S - n)
        assert (counts[r] == load).all() and tokens[r] == n
        if n == 0:
            assert (P[r] == 0).all() and loss[r] == 0
            continue
        fin = np.isfinite(xr)
        top = np.where(fin, xr, -np.inf).max(1)
        low = np.where(fin, xr, np.inf).min(1)
        far = np.where(fin, np.abs(xr), 0.0).max(1) if sigmoid else np.where(fin.any(1), top - low, 0.0)
        c = ((E + 2 * np.minimum(far, 130.0) + 64) * EPS)[:, None]
        den = np.take_along_axis(want["s"], ids, 1).sum(1, keepdims=True) if renorm else np.ones((n, 1))
        lost = sc * TINY / np.where(den > 0, den, 1.0)
        assert (np.abs(w[r][ok] - want["weights"]) <= c * want["weights"] + lost).all()
        tol = (c * want["p"] + TINY / np.where(want["z"] > 0, want["z"], 1.0)).sum(0) + S * EPS * want["P"]
        assert (np.abs(P[r] - want["P"]) <= tol).all()
        b = float(cf) * E / (K * n * n) * want["C"]
        assert abs(loss[r] - want["loss"]) <= (b * tol).sum() + (E + 8) * EPS * abs(want["loss"]) + 1e-36
        g, terms = ref.route_grad(xr, ids, dw[r][ok].astype(np.float64), float(dl[r]), sigmoid, renorm, sc, cf)
        # a score that counts as 0 loses what its own terms would have been
        z = want["z"] if sigmoid else np.ones((n, 1))
        gone = TINY * (float(sc) * np.abs(dw[r][ok]).sum(1, keepdims=True) / np.where(den > 0, den, 1.0) +
                       np.abs(dl[r]) * np.abs(b).max() / np.where(z > 0, z, 1.0))
        assert np.isfinite(d[r]).all()
        assert (np.abs(d[r][ok] - g) <= 4 * c * terms + 2 * gone + 1e-44).all()
    return topk, w, P, loss, d


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("S", [9, 40])
def test_masks_by_token(env, sigmoid, renorm, S):
    """Masks of -infinity and of the type's lowest value beside each other: rows
    with fewer than K experts left, one, none."""
    print(f"[case] masks by token sigmoid={sigmoid} renorm={renorm} S={S}", flush=True)
    rng = np.random.default_rng(16)
    low, high = np.finfo(np.float32).min, np.finfo(np.float32).max
    x = rng.standard_normal((2, S, 70)).astype(np.float32)
    x[rng.random(x.shape) < 0.4] = -np.inf
    x[rng.random(x.shape) < 0.2] = low
    x[0, 3], x[0, 4, 1:], x[1, 7, :66], x[1, 8] = -np.inf, -np.inf, -np.inf, low
    x[1, 5, 3:], x[0, 6, 2], x[1, 2, :] = low, high, 60.0
    check(env, x, 8, sigmoid, renorm)
    if sigmoid:
        check(env, x, 8, sigmoid, renorm, bias=rng.standard_normal(70).astype(np.float32))


@pytest.mark.parametrize("S", [31, 32, 33, 34])
@pytest.mark.parametrize("E,K,sigmoid", [(24, 3, False), (256, 8, True), (320, 40, True)])
def test_around_the_second_launch(env, S, E, K, sigmoid):
    """All outputs at the most tokens of one launch and the fewest of two."""
    print(f"[case] S={S} E={E} K={K} sigmoid={sigmoid}", flush=True)
    rng = np.random.default_rng(S)
    x = (2 * rng.standard_normal((3, S, E))).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if sigmoid else None
    valid = rng.random((3, S)) < 0.8
    valid[2] = False
    valid[1, :-1] = False
    for v in (None, valid):
        check(env, x, K, sigmoid, True, 2.5, bias=bias, valid=v)


@pytest.mark.parametrize("renorm", [False, True])
def test_wide_logits(env, renorm):
    """Logits from -100 to 100: scores of 1 and scores far below."""
    rng = np.random.default_rng(3)
    x = rng.uniform(-100, 100, (2, 50, 96)).astype(np.float32)
    for sigmoid in (False, True):
        print(f"[case] wide logits sigmoid={sigmoid} renorm={renorm}", flush=True)
        check(env, x, 6, sigmoid, renorm)


@pytest.mark.parametrize("K,E", [(2, 8), (1, 5), (8, 128)])
@pytest.mark.parametrize("at", [-60.0, -80.0, -86.0])
def test_gradient_of_small_sigmoids(env, K, E, at):
    """Sigmoids of 1e-26 to 1e-37 throughout, the gradients scaled as a loss
    scaling of 2^16 leaves them: the quotients' gradients are ordinary numbers,
    though the reciprocals of the sums are not."""
    print(f"[case] small sigmoids K={K} E={E} at {at}", flush=True)
    rng = np.random.default_rng(E)
    x = (at + 0.3 * rng.standard_normal((2, 40, E))).astype(np.float32)
    check(env, x, K, True, True, 2.5, dw_scale=65536.0, coef=1.0)


def test_sigmoids_that_count_as_zero(env):
    """Sigmoids below 2^-126 throughout: ids by the logits, all else 0."""
    moon, torch, dev = env
    x = torch.linspace(-120, -90, 40, device=dev).repeat(1, 5, 1).contiguous()
    topk = torch.empty((1, 5, 4), dtype=torch.int32, device=dev)
    w, P, loss = torch.ones((1, 5, 4), device=dev), torch.ones((1, 40), device=dev), torch.ones(1, device=dev)
    c, n, d = torch.empty((1, 40), dtype=torch.int32, device=dev), torch.empty(1, dtype=torch.int32, device=dev), \
        torch.ones_like(x)
    moon.moon_route(x, topk, w, 3, 2.5, tokens_per_expert=c, valid_tokens=n, prob_sums=P, loss=loss, loss_coef=1.0)
    moon.moon_route_backward(x, topk, d, 3, 2.5, d_weights=torch.ones_like(w), tokens_per_expert=c, valid_tokens=n,
                             d_loss=torch.ones(1, device=dev), loss_coef=1.0)
    assert topk[0].tolist() == [[39, 38, 37, 36]] * 5
    assert all(float(a.abs().max()) == 0.0 for a in (w, P, loss, d))
