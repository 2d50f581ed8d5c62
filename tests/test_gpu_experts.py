"""GPU parity of the experts' products over MXFP4 rows and weights against
64-bit products of the same values.

Tolerance of a product: every product of two 4-bit values and their scales is
exact in fp32, so a sum of K of them is off by at most K 2^-23 times the sum of
magnitudes (K additions, each within a step to allow for the matrix core's own
alignment of a block's terms), and rounding to bf16 adds 2^-8 of the value.  The
gated activation passes on the gate's error with a slope of at most 1.1 and the
up product's by silu(G), and adds 32 * 2^-24 of its own."""
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


def random_mx4(rng, shape, cols, mid):
    q = rng.integers(0, 256, (*shape, cols // 2), dtype=np.uint8)
    s = rng.integers(mid - 3, mid + 4, (*shape, cols // 32)).astype(np.uint8)
    return q, s


def close(got, want, bound):
    assert (np.abs(got - want) <= bound + 2.0 ** -8 * np.abs(want) + 1e-30).all()


class Case:
    """Group sizes, MXFP4 rows and weights, and what the products should be."""

    def __init__(self, env, sizes, E, P, K, N, seed, behind=5):
        moon, torch, dev = env
        self.rng = rng = np.random.default_rng(seed)
        self.arrays, self.NvS = ref.plan_arrays(sizes, E, P)
        self.NvS += behind
        self.R, self.EB = self.arrays["cu_seqlens"].shape
        self.E, self.B, self.K, self.N = E, self.EB - E, K, N
        self.kind = ref.row_kinds(self.arrays, self.NvS)
        self.xq, self.xs = random_mx4(rng, (self.R * self.NvS,), K, 126)
        self.xs[self.kind != 1] = 255  # NaN wherever no route is
        self.put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        self.plan = {k: self.put(v) for k, v in self.arrays.items()}
        self.ws = [self.weight() for _ in range(2)]
        self.row_w = rng.standard_normal(self.R * self.NvS).astype(np.float32)
        self.row_w[self.kind != 1] = np.nan

    def weight(self):
        eq, es = random_mx4(self.rng, (self.E, self.N), self.K, 122)
        sq, ss = random_mx4(self.rng, (self.R, self.B, self.N), self.K, 122)
        return eq, es, sq, ss

    def products(self, w):
        """(y, sum of magnitudes) [R*NvS, N]."""
        y = np.zeros((self.R, self.NvS, self.N))
        a = np.zeros_like(y)
        x = ref.mx4_values(self.xq, np.where(self.xs == 255, 127, self.xs)).reshape(self.R, self.NvS, -1)
        for u, g, b, e, _ in ref.spans(self.arrays):
            q, s = (w[0][g], w[1][g]) if g < self.E else (w[2][u, g - self.E], w[3][u, g - self.E])
            v = ref.mx4_values(q, s)
            y[u, b:e] = x[u, b:e] @ v.T
            a[u, b:e] = np.abs(x[u, b:e]) @ np.abs(v).T
        return y.reshape(-1, self.N), a.reshape(-1, self.N)

    def dev(self, w):
        return tuple(self.put(a) for a in w)

    def check_rows(self, y, want, bound):
        k = self.kind
        close(y[k == 1], want[k == 1], bound[k == 1])
        assert (y[k == 2] == 0).all()
        assert (y[k == 0] == 77).all()

    def run(self, env, swiglu, weighted=False):
        moon, torch, dev = env
        y = torch.full((self.R * self.NvS, self.N), 77.0, dtype=torch.bfloat16, device=dev)
        xq, xs = self.put(self.xq), self.put(self.xs)
        if swiglu:
            moon.moon_expert_swiglu_mx4(self.plan, xq, xs, self.dev(self.ws[0]), self.dev(self.ws[1]), y,
                                        row_weights=self.put(self.row_w) if weighted else None)
        else:
            moon.moon_expert_gemm_mx4(self.plan, xq, xs, self.dev(self.ws[0]), y)
        torch.cuda.synchronize()
        return y.double().cpu().numpy()

    def check(self, env):
        G, aG = self.products(self.ws[0])
        U, aU = self.products(self.ws[1])
        step = self.K * 2.0 ** -23
        self.check_rows(self.run(env, False), G, step * aG)
        for weighted in (False, True):
            c = np.where(self.kind == 1, self.row_w, 1.0).astype(np.float64)[:, None] if weighted else 1.0
            want = c * ref.silu(G) * U
            eG, eU = step * aG, step * aU
            bound = np.abs(c) * (1.1 * eG * (np.abs(U) + eU) + np.abs(ref.silu(G)) * eU) + \
                32 * 2.0 ** -24 * np.abs(want)
            self.check_rows(self.run(env, True, weighted), want, bound)


def own(R, E, B, rows, slots=None):
    """Sizes [R, E+B]: rank u's own experts hold rows[...] in turn."""
    n = np.zeros((R, E + B), np.int64)
    Eg = E // R
    it = iter(rows)
    for u in range(R):
        for i in range(Eg):
            n[u, u * Eg + i] = next(it)
        for j, k in enumerate((slots or [[]] * R)[u]):
            n[u, E + j] = k
    return n


@pytest.mark.parametrize("label,R,E,B,P,rows,slots,K,N", [
    ("one row", 1, 1, 1, 1, [1], None, 32, 8),
    ("edges of 16", 1, 6, 2, 1, [0, 1, 15, 16, 17, 0], None, 96, 40),
    ("two ranks, slots", 2, 4, 2, 8, [3, 0, 9, 64], [[5, 0], [0, 0]], 544, 72),
    ("K 512", 2, 2, 1, 16, [33, 65], [[0], [1]], 512, 24),
    ("K 2080", 1, 2, 2, 4, [7, 70], [[0, 0]], 2080, 264),
    ("many rows", 2, 4, 2, 128, [130, 300, 1, 511], [[64, 0], [257, 2]], 256, 128),
    ("wide", 1, 2, 1, 1, [5, 260], None, 1024, 1032),
    ("long", 1, 1, 1, 1, [3], None, 8192, 16),
    ("more slots than experts", 2, 2, 4, 1, [3, 4], [[2, 0, 0, 0], [0, 0, 0, 0]], 64, 32),
    ("large tiles", 2, 4, 2, 16, [700, 0, 513, 256], [[255, 0], [31, 0]], 1056, 520),
    ("one large group among small ones", 1, 16, 1, 1, [40] + [1] * 15, None, 512, 72),
    ("the same, ragged K", 1, 16, 1, 1, [1] * 15 + [33], None, 608, 40),
    ("whole turns, odd number", 2, 16, 2, 4, [2, 3] * 8, [[1, 0], [5, 0]], 1536, 136),
    ("middling groups", 2, 4, 1, 8, [40, 70, 64, 17], [[20], [0]], 1024, 264),
    ("middling, six steps", 2, 4, 1, 8, [40, 70, 64, 17], [[20], [0]], 1536, 64),
    ("tiles, one turn", 1, 2, 1, 1, [257, 300], None, 512, 264),
    ("tiles, two turns", 2, 4, 1, 16, [300, 513, 0, 256], [[190], [0]], 1024, 256),
    ("tiles, three turns", 1, 1, 1, 1, [600], None, 1536, 392),
    ("tiles, a few columns", 1, 1, 1, 1, [1000], None, 512, 8),
    ("tiles, the shortest K", 1, 2, 1, 1, [200, 129], None, 32, 48),
])
def test_products(env, label, R, E, B, P, rows, slots, K, N):
    say(f"[case] products {label}: R={R} E={E} B={B} P={P} K={K} N={N}")
    Case(env, own(R, E, B, rows, slots), E, P, K, N, seed=K + N).check(env)


def test_lane_layout(env):
    """Single ones: row r holds a one at k = 37 r + 5 (mod K), so every output
    names one weight and one scale exactly."""
    moon, torch, dev = env
    c = Case(env, own(1, 1, 1, [64]), 1, 1, 512, 64, seed=1)
    k = (37 * np.arange(c.NvS) + 5) % 512
    codes = np.zeros((c.NvS, 512), np.uint8)
    codes[np.arange(c.NvS), k] = 2  # 1.0
    c.xq, c.xs = ref.pack4(codes), np.full((c.NvS, 16), 127, np.uint8)
    y = c.run(env, False)
    w = ref.mx4_values(c.ws[0][0][0], c.ws[0][1][0])
    want = torch.from_numpy(w[:, k[:64]].T.copy()).bfloat16().double().numpy()
    assert (y[:64] == want).all()


@pytest.mark.parametrize("rows", [(40, 20), (300, 260), (3, 2)])
@pytest.mark.parametrize("K", [320, 512])
def test_nan_scales_reach_their_outputs_only(env, rows, K):
    """A NaN block of one row or one weight row makes that row's or column's
    outputs NaN and no others."""
    c = Case(env, own(1, 2, 1, rows), 2, 1, K, 48, seed=2)
    c.xs[rows[0] - 1, 3] = 255
    c.ws[0][1][1, 33, 9] = 255
    y = c.run(env, False)
    bad = np.zeros(y.shape, bool)
    bad[rows[0] - 1] = True
    bad[rows[0]:sum(rows), 33] = True
    assert (np.isnan(y) == bad).all()


@pytest.mark.parametrize("rows", [(5, 20), (300, 130)])
@pytest.mark.parametrize("up,down", [(250, 4), (4, 250), (254, 0), (0, 254)])
def test_scales_at_their_ends(env, rows, up, down):
    """Scales of 2^123 against 2^-123, and of 2^127 against 2^-127: the products
    are ordinary numbers, and stay exact."""
    c = Case(env, own(1, 2, 1, rows), 2, 1, 544, 40, seed=6)
    c.xs[c.kind == 1] = up
    for a in c.ws[0][1::2]:
        a[:] = down
    y, mag = c.products(c.ws[0])
    c.check_rows(c.run(env, False), y, c.K * 2.0 ** -23 * mag)


def test_rows_beyond_32_bit_offsets(env):
    """A window of 2.4e9 outputs (4.8 GB): rows at both ends of it."""
    moon, torch, dev = env
    K, N, rows = 64, 8192, 300000
    arrays, NvS = ref.plan_arrays([[rows - 7, 5, 0]], 2, 1)
    plan = {k: torch.from_numpy(v).to(dev) for k, v in arrays.items()}
    g = torch.Generator(device=dev).manual_seed(1)
    rnd = lambda lo, hi, *n: torch.randint(lo, hi, n, generator=g, device=dev, dtype=torch.uint8)  # noqa: E731
    xq, xs = rnd(0, 255, NvS, K // 2), rnd(124, 129, NvS, K // 32)
    w = (rnd(0, 255, 2, N, K // 2), rnd(120, 125, 2, N, K // 32), rnd(0, 255, 1, 1, N, K // 2),
         rnd(120, 125, 1, 1, N, K // 32))
    y = torch.full((NvS, N), 77.0, dtype=torch.bfloat16, device=dev)
    moon.moon_expert_gemm_mx4(plan, xq, xs, w, y)
    values = lambda q, s: ref.mx4_values(q.cpu().numpy(), s.cpu().numpy())  # noqa: E731
    for at, e in ((slice(0, 9), 0), (slice(rows - 20, rows - 7), 0), (slice(rows - 7, rows - 2), 1)):
        x, v = values(xq[at], xs[at]), values(w[0][e], w[1][e])
        close(y[at].double().cpu().numpy(), x @ v.T, K * 2.0 ** -23 * (np.abs(x) @ np.abs(v).T))


def test_failed_plan_writes_nothing(env):
    c = Case(env, own(1, 2, 1, [40, 300]), 2, 16, 128, 64, seed=3)
    c.plan["status"].fill_(2)
    assert (c.run(env, False) == 77).all() and (c.run(env, True) == 77).all()


def test_repeats_and_graph(env):
    """Equal bits call after call, on a side stream and in replays between
    eager calls on other rows."""
    moon, torch, dev = env
    for rows in ([5, 3, 0, 20], [900, 300, 0, 260]):
        c = Case(env, own(2, 4, 1, rows), 4, 8, 416, 96, seed=4)
        xq, xs = c.put(c.xq), c.put(c.xs)
        other = c.put(np.roll(c.xq, 5, 1))
        gate, up = c.dev(c.ws[0]), c.dev(c.ws[1])
        shape = (c.R * c.NvS, c.N)
        h, y = (torch.zeros(shape, dtype=torch.bfloat16, device=dev) for _ in range(2))

        def step(q, h, y, stream=None):
            moon.moon_expert_swiglu_mx4(c.plan, q, xs, gate, up, h, stream=stream)
            moon.moon_expert_gemm_mx4(c.plan, q, xs, gate, y, stream=stream)

        want = []
        for q in (xq, other):
            step(q, h, y)
            want.append((h.clone(), y.clone()))
        side = torch.cuda.Stream(device=dev)
        h.zero_()
        side.wait_stream(torch.cuda.current_stream())
        step(xq, h, y, stream=side)
        side.synchronize()
        assert torch.equal(h, want[0][0]) and torch.equal(y, want[0][1])
        q = xq.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(q, h, y)
        for i in (1, 0, 1):
            q.copy_(other if i else xq)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(h, want[i][0]) and torch.equal(y, want[i][1])
            step(other, torch.zeros_like(h), torch.zeros_like(y))


def test_refusals(env):
    moon, torch, dev = env
    c = Case(env, own(1, 2, 1, [4, 3]), 2, 1, 64, 16, seed=5)
    y = torch.zeros((c.NvS, 16), dtype=torch.bfloat16, device=dev)
    ok = dict(plan=c.plan, xq=c.put(c.xq), xs=c.put(c.xs), weight=c.dev(c.ws[0]), y=y)
    moon.moon_expert_gemm_mx4(**ok)
    w = ok["weight"]
    for bad in (dict(xq=ok["xq"][:, :16]), dict(xs=ok["xs"][:, :1].contiguous()), dict(y=y.float()),
                dict(y=y[:-1]), dict(weight=(w[0][:1], *w[1:])), dict(weight=(*w[:2], w[2].float(), w[3])),
                dict(weight=(w[0].cpu(), *w[1:])), dict(xq=ok["xq"][0])):
        with pytest.raises(ValueError):
            moon.moon_expert_gemm_mx4(**{**ok, **bad})
    n12 = tuple(t[..., :12, :].contiguous() for t in w)  # 12 outputs: no multiple of 8
    with pytest.raises(moon.MoonError):
        moon.moon_expert_gemm_mx4(**{**ok, "weight": n12, "y": y[:, :12].contiguous()})


@pytest.mark.parametrize("rows", [3, 20, 300])
@pytest.mark.parametrize("K", [512, 544])
def test_padding_without_routes(env, rows, K):
    """Groups of nothing but padding, which only a caller's own arrays have: the
    first, one between others and the last, in every kernel."""
    say(f"[case] groups of padding only, rows={rows} K={K}")
    c = Case(env, own(2, 8, 1, [rows] * 8, [[rows], [rows]]), 8, 4, K, 72, seed=rows)
    cu, zfr = c.arrays["cu_seqlens"], c.arrays["zero_fill_ranges"]
    for u, g in [(0, 0), (0, 2), (1, 5), (1, 8)]:
        zfr[u, g, 0] = cu[u, g - 1] if g > 0 else 0
    c.kind = ref.row_kinds(c.arrays, c.NvS)
    assert (c.kind == 2).sum() >= 4 * rows
    c.xs[c.kind != 1], c.row_w[c.kind != 1] = 255, np.nan
    c.plan = {k: c.put(v) for k, v in c.arrays.items()}
    c.check(env)


@pytest.mark.parametrize("rows", [3, 20, 300])
@pytest.mark.parametrize("off", [1, 4])
def test_scales_anywhere(env, rows, off):
    """Scale bytes may start at any address, whole turns of them too."""
    moon, torch, dev = env
    say(f"[case] scales {off} bytes off, rows={rows}")
    c = Case(env, own(1, 4, 1, [rows] * 4, [[rows]]), 4, 1, 512, 72, seed=rows + off)

    def moved(a):
        buf = torch.full((a.size + 16,), 255, dtype=torch.uint8, device=dev)
        buf[off:off + a.size] = c.put(a).view(-1)
        return buf[off:off + a.size].view(a.shape)

    G, bound = c.products(c.ws[0])
    eq, es, sq, ss = c.ws[0]
    for xs, w in ((moved(c.xs), c.dev(c.ws[0])), (c.put(c.xs), (c.put(eq), moved(es), c.put(sq), c.put(ss))),
                  (c.put(c.xs), (c.put(eq), c.put(es), c.put(sq), moved(ss)))):
        y = torch.full((c.NvS, 72), 77.0, dtype=torch.bfloat16, device=dev)
        moon.moon_expert_gemm_mx4(c.plan, c.put(c.xq), xs, w, y)
        torch.cuda.synchronize()
        c.check_rows(y.double().cpu().numpy(), G, 512 * 2.0 ** -23 * bound)
