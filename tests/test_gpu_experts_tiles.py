"""The tile kernels of the experts' products from one tile to the next: far more
tiles than workgroups, every output compared with products in 64 bits.

Bounds as for the other products: a sum of K exact products is off by at most
K 2^-23 of the sum of magnitudes and rounding to bf16 by 2^-8 of the value; the
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


def sizes(R, E, B, rng):
    """Rows of every group: a few past a multiple of 256 in most, some exact,
    some small, some none."""
    n = np.zeros((R, E + B), np.int64)
    Eg = E // R
    some = [257, 300, 0, 513, 256, 7, 259, 512, 1, 770]
    for u in range(R):
        for i, k in enumerate(rng.permutation(np.resize(some, Eg + B))):
            n[u, u * Eg + i if i < Eg else E + i - Eg] = k
    return n


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K", [512, 1024, 1536, 1056, 96])
def test_tile_after_tile(env, K, swiglu):
    moon, torch, dev = env
    R, E, B, P = 2, 32, 4, 8
    N = 1032 if swiglu else 2312  # 9 and 10 tiles wide, the last of 8 outputs
    rng = np.random.default_rng(K + swiglu)
    n = sizes(R, E, B, rng)
    arrays, NvS = ref.plan_arrays(n, E, P)
    NvS += 5
    cu, zfr = arrays["cu_seqlens"], arrays["zero_fill_ranges"]
    for u, g in [(0, 1), (0, E + 1), (1, 20)]:  # and groups of nothing but padding
        zfr[u, g, 0] = cu[u, g - 1]
    kind = ref.row_kinds(arrays, NvS)
    groups = [(u, g, a, b) for u, g, a, b, _ in ref.spans(arrays) if b > a]
    tiles = sum((b - a + 255) // 256 for _, _, a, b in groups) * ((N + 255 - 128 * swiglu) // (256 - 128 * swiglu))
    print(f"[case] tiles after tiles K={K} N={N} swiglu={swiglu}: {tiles} tiles", flush=True)
    assert tiles > 2 * 256
    gen = torch.Generator(device=dev).manual_seed(K)
    u8 = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen, device=dev, dtype=torch.uint8)  # noqa: E731
    rows = R * NvS
    live = torch.from_numpy(kind == 1).to(dev)
    pad = torch.from_numpy(kind == 2).to(dev)
    xq, xs = u8(0, 256, rows, K // 2), u8(123, 130, rows, K // 32)
    xs[~live] = 255
    ws = [(u8(0, 256, E, N, K // 2), u8(119, 126, E, N, K // 32), u8(0, 256, R, B, N, K // 2),
           u8(119, 126, R, B, N, K // 32)) for _ in range(1 + swiglu)]
    rw = torch.randn((rows,), generator=gen, device=dev)
    rw[~live] = float("nan")
    plan = {k: torch.from_numpy(v).to(dev) for k, v in arrays.items()}
    y = torch.full((rows, N), 77.0, dtype=torch.bfloat16, device=dev)
    if swiglu:
        moon.moon_expert_swiglu_mx4(plan, xq, xs, ws[0], ws[1], y, row_weights=rw)
    else:
        moon.moon_expert_gemm_mx4(plan, xq, xs, ws[0], y)
    torch.cuda.synchronize()
    assert bool((y[pad] == 0).all()) and bool((y[~live & ~pad] == 77).all())
    grid = torch.tensor(np.concatenate([ref.E2M1, -ref.E2M1]), device=dev)

    def values(q, s):
        v = grid[torch.stack([q & 15, q >> 4], -1).flatten(-2).int()]
        return (v.view(v.shape[0], -1, 32) * torch.exp2(s.double() - 127)[..., None]).flatten(1)

    step = K * 2.0 ** -23
    for u, g, a, b in groups:
        at = slice(u * NvS + a, u * NvS + b)
        x = values(xq[at], xs[at])
        prod = []
        for eq, es, sq, ss in ws:
            w = values(eq[g], es[g]) if g < E else values(sq[u, g - E], ss[u, g - E])
            prod.append((x @ w.t().contiguous(), step * (x.abs() @ w.abs().t().contiguous())))
        if swiglu:
            (G, eG), (U, eU) = prod
            act, c = G / (1 + torch.exp(-G)), rw[at, None].double()
            want = c * act * U
            bound = c.abs() * (1.1 * eG * (U.abs() + eU) + act.abs() * eU) + 32 * 2.0 ** -24 * want.abs()
        else:
            want, bound = prod[0]
        assert bool(((y[at].double() - want).abs() <= bound + 2.0 ** -8 * want.abs() + 1e-30).all()), (u, g)
