"""The routing and expert operators together with plan, dispatch, weight
prefetch, combine and gradient reduction, as a layer runs them.

Serving: route -> plan -> dispatch -> 4-bit rows -> prefetch of 4-bit weights ->
gate/up product with activation -> 4-bit rows -> down product -> combine.
Training: route -> plan -> dispatch -> the caller's products -> activation with
8-bit saved inputs -> combine, and back: dispatch of the gradient along the same
plan -> activation gradient -> weight gather of the combine -> router gradient.

Every stage is compared token by token in 64 bits through the experts that the
router chose (dst gives a route's row), never through the group arrays that the
kernels walk."""
import numpy as np
import pytest

import operator_refs as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import combine_balanced_planning_amd as moon
    return moon, torch, torch.device("cuda", 0)


def say(*a):
    print(*a, flush=True)


class Layer:
    """Sizes, a planned batch from the router, and what maps rows to experts."""

    def __init__(self, env, R, E, K, S, H, B, P, sigmoid, seed, noalloc=False, skew=2.0):
        moon, torch, dev = env
        self.R, self.E, self.K, self.S, self.H = R, E, K, S, H
        g = self.g = torch.Generator(device=dev).manual_seed(seed)
        self.logits = torch.randn((R, S, E), generator=g, device=dev) - \
            skew * torch.log1p(torch.arange(E, device=dev).float())
        self.valid = torch.rand((R, S), generator=g, device=dev) < 0.9
        self.hidden = torch.randn((R, S, H), generator=g, device=dev).bfloat16()
        self.hidden[~self.valid] = 0
        self.flags = moon.MOON_ROUTE_RENORM | (moon.MOON_ROUTE_SIGMOID if sigmoid else 0)
        self.topk = torch.empty((R, S, K), dtype=torch.int32, device=dev)
        self.weights = torch.empty((R, S, K), device=dev)
        self.tpe = torch.empty((R, E), dtype=torch.int32, device=dev)
        self.ntok = torch.empty((R,), dtype=torch.int32, device=dev)
        self.psum, self.loss = torch.empty((R, E), device=dev), torch.empty((R,), device=dev)
        moon.moon_route(self.logits, self.topk, self.weights, self.flags, 1.0, valid=self.valid,
                        tokens_per_expert=self.tpe, valid_tokens=self.ntok, prob_sums=self.psum,
                        loss=self.loss, loss_coef=0.01)
        self.ctx = moon.moon_ctx_create(R, E, K, S, H, B, P)
        self.plan = moon.moon_plan_create(self.ctx)
        moon.moon_plan(self.ctx, self.topk, self.tpe, self.plan)
        assert moon.moon_plan_status(self.plan) == moon.MOON_OK
        moon.moon_dispatch(self.ctx, self.plan, self.hidden, self.weights)
        self.win, self.wwin = moon.window_tensors(self.ctx)
        self.rows = R * self.ctx.NvS
        self.groups = self.plan
        if noalloc:  # the operators take the caller's own plan arrays as well
            shapes, NvS, Bx = moon.plan_array_shapes(R, E, K, S, B, P)
            self.groups = {k: torch.empty(s, dtype=torch.int32, device=dev) for k, s in shapes.items()}
            moon.moon_plan_noalloc(R, E, K, S, H, B, P, self.topk, self.tpe, self.groups)
            assert NvS == self.ctx.NvS and Bx == self.ctx.B
        dst = moon.plan_tensors(self.plan)["dst"].cpu().numpy().reshape(R, S, K).astype(np.int64)
        self.row = np.where(dst >= 0, dst, -dst - 1)          # [R, S, K]
        self.expert = self.topk.cpu().numpy()
        self.used = int((moon.plan_tensors(self.plan)["experts_to_copy"] >= 0).sum())

    def close(self, env):
        env[0].moon_plan_destroy(self.plan)
        env[0].moon_ctx_destroy(self.ctx)


def within(got, want, bound):
    assert (np.abs(got - want) <= bound + 2.0 ** -8 * np.abs(want) + 1e-30).all()


@pytest.mark.parametrize("R,E,K,S,H,F,B,P,sigmoid,noalloc", [
    (4, 16, 4, 96, 128, 96, 4, 8, True, False),
    (2, 8, 2, 300, 256, 64, 4, 16, False, True),
    (8, 32, 4, 3, 96, 64, 4, 1, False, False),   # three tokens a rank
    (1, 4, 4, 700, 512, 128, 2, 128, True, True),
])
def test_serving_layer(env, R, E, K, S, H, F, B, P, sigmoid, noalloc):
    moon, torch, dev = env
    say(f"[case] serving layer R={R} E={E} K={K} S={S} H={H} F={F} P={P}")
    L = Layer(env, R, E, K, S, H, B, P, sigmoid, seed=S + H, noalloc=noalloc)
    try:
        u8 = lambda *n: torch.zeros(n, dtype=torch.uint8, device=dev)  # noqa: E731
        full, packed = {}, {}
        for name, n, k in (("gate", F, H), ("up", F, H), ("down", H, F)):
            w = (torch.randn((E, n, k), generator=L.g, device=dev) * k ** -0.5).bfloat16()
            q, s = u8(E, n, k // 2), u8(E, n, k // 32)
            moon.moon_mx4_quantize(w, q, s)
            sq, ss = u8(R, L.ctx.B, n, k // 2), u8(R, L.ctx.B, n, k // 32)
            # codes and scales go into the slots like any other weight (rows of 16 bytes)
            flat = lambda t, lead: t.view(*t.shape[:lead], -1)  # noqa: E731
            pad = -flat(s, 1).shape[1] % 16
            se = torch.nn.functional.pad(flat(s, 1), (0, pad))
            sl = torch.nn.functional.pad(flat(ss, 2), (0, pad))
            moon.moon_prefetch_weight(L.ctx, L.plan, [flat(q, 1), se.contiguous()], [flat(sq, 2), sl])
            ss = sl[..., :n * k // 32].reshape(ss.shape).contiguous()
            packed[name] = (q, s, sq, ss)
            full[name] = ref.mx4_values(q.cpu().numpy(), s.cpu().numpy())
        xq, xs = u8(L.rows, H // 2), u8(L.rows, H // 32)
        h = torch.zeros((L.rows, F), dtype=torch.bfloat16, device=dev)
        hq, hs = u8(L.rows, F // 2), u8(L.rows, F // 32)
        y = torch.zeros((L.rows, H), dtype=torch.bfloat16, device=dev)
        out = torch.empty((R, S, H), dtype=torch.bfloat16, device=dev)
        moon.moon_mx4_quantize(L.win, xq, xs, plan=L.groups)
        moon.moon_expert_swiglu_mx4(L.groups, xq, xs, packed["gate"], packed["up"], h, row_weights=L.wwin)
        moon.moon_mx4_quantize(h, hq, hs, plan=L.groups)
        moon.moon_expert_gemm_mx4(L.groups, hq, hs, packed["down"], y)
        moon.moon_combine(L.ctx, L.plan, y, None, 0, out)
        torch.cuda.synchronize()
        # a route's row is its token's, quantised
        hid = L.hidden.double().cpu().numpy()
        q, s = ref.mx4(hid)
        row, ex = L.row.reshape(-1), L.expert.reshape(-1)
        tok = np.arange(R * S * K) // K
        assert (xq.cpu().numpy()[row] == q.reshape(R * S, -1)[tok]).all()
        assert (xs.cpu().numpy()[row] == s.reshape(R * S, -1)[tok]).all()
        x = ref.mx4_values(q, s).reshape(R * S, H)[tok]
        c = L.weights.double().cpu().numpy().reshape(-1)
        got_h, got_y = h.double().cpu().numpy(), y.double().cpu().numpy()
        hv = ref.mx4_values(hq.cpu().numpy(), hs.cpu().numpy())
        wq, ws = ref.mx4(got_h[row])
        assert (hq.cpu().numpy()[row] == wq).all() and (hs.cpu().numpy()[row] == ws).all()
        for e in range(E):
            i = np.flatnonzero(ex == e)
            G, U = x[i] @ full["gate"][e].T, x[i] @ full["up"][e].T
            aG, aU = np.abs(x[i]) @ np.abs(full["gate"][e]).T, np.abs(x[i]) @ np.abs(full["up"][e]).T
            eG, eU = H * 2.0 ** -23 * aG, H * 2.0 ** -23 * aU
            want = c[i, None] * ref.silu(G) * U
            within(got_h[row[i]], want, c[i, None] * (1.1 * eG * (np.abs(U) + eU) + np.abs(ref.silu(G)) * eU) +
                   32 * 2.0 ** -24 * np.abs(want))
            hd = hv[row[i]]
            within(got_y[row[i]], hd @ full["down"][e].T,
                   F * 2.0 ** -23 * (np.abs(hd) @ np.abs(full["down"][e]).T))
        # the combine adds a token's K rows in fp32, in order: K 2^-24 of their magnitudes
        per = got_y[row].reshape(R, S, K, H)
        within(out.double().cpu().numpy(), per.sum(2), K * 2.0 ** -24 * np.abs(per).sum(2))
        assert R == 1 or L.used > 0
    finally:
        L.close(env)


@pytest.mark.parametrize("R,E,K,S,H,F,B,P,sigmoid", [(4, 8, 2, 120, 64, 64, 2, 8, False),
                                                     (2, 6, 3, 77, 96, 32, 3, 5, True)])
def test_training_layer(env, R, E, K, S, H, F, B, P, sigmoid):
    """The gradient of the logits through the whole layer against 64 bits; the
    caller's products (gate/up and down) are plain matrix products here."""
    moon, torch, dev = env
    say(f"[case] training layer R={R} E={E} K={K} S={S} H={H} F={F} P={P}")
    L = Layer(env, R, E, K, S, H, B, P, sigmoid, seed=S)
    try:
        w1 = torch.randn((E, 2 * F, H), generator=L.g, device=dev) * H ** -0.5
        w2 = torch.randn((E, H, F), generator=L.g, device=dev) * F ** -0.5
        row, ex = torch.from_numpy(L.row.reshape(-1)).to(dev), L.topk.reshape(-1)
        bf = lambda n: torch.zeros((L.rows, n), dtype=torch.bfloat16, device=dev)  # noqa: E731

        def product(x, w, n):
            """Rows times their experts' weights, by the caller."""
            o = bf(n)
            for e in range(E):
                i = row[ex == e]
                o[i] = (x[i].float() @ w[e].T).bfloat16()
            return o

        gu = product(L.win, w1, 2 * F)
        h, saved = bf(F), torch.zeros((L.rows, 2 * F), dtype=torch.uint8, device=dev)
        scales = torch.zeros((L.rows, 2 * F // 32), dtype=torch.uint8, device=dev)
        moon.moon_swiglu_save8(L.plan, gu, h, saved, scales, row_weights=L.wwin)
        y = product(h, w2, H)
        out = torch.empty((R, S, H), dtype=torch.bfloat16, device=dev)
        moon.moon_combine(L.ctx, L.plan, y, None, 0, out)
        # back: the gradient travels along the same plan
        dout = torch.randn((R, S, H), generator=L.g, device=dev).bfloat16()
        dy = bf(H)
        moon.moon_dispatch(L.ctx, L.plan, dout, hidden_out=dy)
        dh = product(dy, w2.transpose(1, 2), F)
        dgu, dw = bf(2 * F), torch.zeros((L.rows,), device=dev)
        moon.moon_swiglu_grad8(L.plan, dh, saved, scales, dgu, row_weights=L.wwin, d_row_weights=dw)
        dx = product(dgu, w1.transpose(1, 2), H)
        dhid = torch.empty((R, S, H), dtype=torch.bfloat16, device=dev)
        dweights = torch.empty((R, S, K), device=dev)
        moon.moon_combine(L.ctx, L.plan, dx, dw, 0, dhid, dweights)
        dl = torch.full((R,), 3.0, device=dev)
        dlog = torch.empty_like(L.logits)
        moon.moon_route_backward(L.logits, L.topk, dlog, L.flags, 1.0, valid=L.valid, d_weights=dweights,
                                 tokens_per_expert=L.tpe, valid_tokens=L.ntok, d_loss=dl, loss_coef=0.01)
        torch.cuda.synchronize()
        n64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        r, e = row.cpu().numpy(), ex.cpu().numpy()
        g64 = n64(gu)[r]
        s = ref.mx_scale(g64, 8)
        v = ref.mx_values(ref.mx_codes(g64, s, 8), s, 8)
        d, c = n64(dh)[r], n64(L.weights).reshape(-1, 1)
        act = ref.silu(v[:, :F])
        terms = d * act * v[:, F:]
        want_dw = terms.sum(1).reshape(R, S, K)
        # F terms summed in fp32, each off by 32 units of 2^-24
        tol = (F + 32) * 2.0 ** -24 * np.abs(terms).sum(1).reshape(R, S, K)
        assert (np.abs(n64(dweights) - want_dw) <= tol + 1e-30).all()
        want = np.concatenate([c * d * v[:, F:] * ref.silu_slope(v[:, :F]), c * d * act], 1)
        big = np.concatenate([np.abs(c * d * v[:, F:]) * (1 + np.abs(v[:, :F])), np.abs(c * d * v[:, :F])], 1)
        within(n64(dgu)[r], want, 32 * 2.0 ** -24 * big)
        valid = L.valid.cpu().numpy()
        for u in range(R):
            ok = valid[u]
            x = n64(L.logits)[u][ok]
            span = 2 * max(np.ptp(x, axis=1).max(), np.abs(x).max())
            g, terms = ref.route_grad(x, L.expert[u][ok], n64(dweights)[u][ok], 3.0, sigmoid, True, 1.0,
                                      np.float32(0.01))
            got = n64(dlog)[u]
            assert (got[~ok] == 0).all()
            assert (np.abs(got[ok] - g) <= 4 * (E + span + 64) * 2.0 ** -24 * terms + 1e-36).all()
        # the combine sums K rows of the hidden's gradient
        per = n64(dx)[r].reshape(R, S, K, H)
        within(n64(dhid), per.sum(2), K * 2.0 ** -24 * np.abs(per).sum(2))
    finally:
        L.close(env)


def test_serving_layer_in_a_graph(env):
    """The whole serving layer captured once and replayed on other logits and
    tokens: every replay equals the eager layer bit for bit."""
    moon, torch, dev = env
    R, E, K, S, H, F, B, P = 4, 16, 4, 40, 128, 64, 4, 8
    g = torch.Generator(device=dev).manual_seed(11)
    u8 = lambda *n: torch.zeros(n, dtype=torch.uint8, device=dev)  # noqa: E731
    ctx = moon.moon_ctx_create(R, E, K, S, H, B, P)
    plan = moon.moon_plan_create(ctx)
    try:
        win, wwin = moon.window_tensors(ctx)
        rows = R * ctx.NvS
        w = {}
        for name, n, k in (("gate", F, H), ("up", F, H), ("down", H, F)):
            q, s = u8(E, n, k // 2), u8(E, n, k // 32)
            moon.moon_mx4_quantize((torch.randn((E, n, k), generator=g, device=dev) * k ** -0.5), q, s)
            w[name] = (q, s, u8(R, B, n, k // 2), u8(R, B, n, k // 32))
        sets = [(torch.randn((R, S, E), generator=g, device=dev),
                 torch.randn((R, S, H), generator=g, device=dev).bfloat16()) for _ in range(3)]
        logits, hidden = sets[0][0].clone(), sets[0][1].clone()
        topk = torch.zeros((R, S, K), dtype=torch.int32, device=dev)
        wt, tpe = torch.zeros((R, S, K), device=dev), torch.zeros((R, E), dtype=torch.int32, device=dev)
        xq, xs, hq, hs = u8(rows, H // 2), u8(rows, H // 32), u8(rows, F // 2), u8(rows, F // 32)
        h = torch.zeros((rows, F), dtype=torch.bfloat16, device=dev)
        y = torch.zeros((rows, H), dtype=torch.bfloat16, device=dev)

        def layer(logits, hidden, out):
            moon.moon_route(logits, topk, wt, moon.MOON_ROUTE_RENORM, tokens_per_expert=tpe)
            moon.moon_plan(ctx, topk, tpe, plan)
            moon.moon_dispatch(ctx, plan, hidden, wt)
            for q, s, sq, ss in w.values():
                moon.moon_prefetch_weight(ctx, plan, [q.view(E, -1), s.view(E, -1)],
                                          [sq.view(R, B, -1), ss.view(R, B, -1)])
            moon.moon_mx4_quantize(win, xq, xs, plan=plan)
            moon.moon_expert_swiglu_mx4(plan, xq, xs, w["gate"], w["up"], h, row_weights=wwin)
            moon.moon_mx4_quantize(h, hq, hs, plan=plan)
            moon.moon_expert_gemm_mx4(plan, hq, hs, w["down"], y)
            moon.moon_combine(ctx, plan, y, None, 0, out)

        out = torch.zeros((R, S, H), dtype=torch.bfloat16, device=dev)
        want = []
        for lg, hd in sets:
            layer(lg, hd, out)
            assert moon.moon_plan_status(plan) == moon.MOON_OK
            want.append(out.clone())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer(logits, hidden, out)
        other = torch.zeros_like(out)
        for i in (1, 2, 0, 2):
            logits.copy_(sets[i][0])
            hidden.copy_(sets[i][1])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out.view(torch.int16), want[i].view(torch.int16)), i
            layer(*sets[(i + 1) % 3], other)
    finally:
        moon.moon_plan_destroy(plan)
        moon.moon_ctx_destroy(ctx)
