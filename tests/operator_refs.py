"""Plain 64-bit implementations of the routing and expert operators, written
from their formulas, for the tests (numpy only; nothing of the library)."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)
                 if not (e == 15 and m == 7)])


# ---- routing ----
def scores(x, sigmoid):
    """Scores of logits x [T, E] (float64): a sigmoid, or a softmax in which
    -inf masks and a row of nothing else is all zeros."""
    if sigmoid:
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    m = x.max(1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    e = np.exp(x - m)
    z = e.sum(1, keepdims=True)
    return e / np.where(z == 0, 1.0, z)


def select(key, K):
    """Ids of the K largest keys, descending, lower id first among equals."""
    T, E = key.shape
    if T == 0:
        return np.zeros((0, K), np.int64)
    return np.stack([np.lexsort((np.arange(E), -key[t]))[:K] for t in range(T)])


def route(x, K, sigmoid=False, renorm=False, scale=1.0, bias=None, coef=0.0, ids=None):
    """One rank's valid tokens x [n, E]: dict of ids, weights, C, P and loss."""
    n, E = x.shape
    s = scores(x, sigmoid)
    if ids is None:
        key = x if bias is None else np.where(np.isneginf(x), -np.inf, s + bias)
        ids = select(key, K)
    sel = np.take_along_axis(s, ids, 1)
    den = sel.sum(1, keepdims=True) if renorm else np.ones((n, 1))
    w = scale * sel / np.where(den == 0, 1.0, den)
    z = s.sum(1, keepdims=True)
    p = s / np.where(z == 0, 1.0, z)
    C = np.bincount(ids.reshape(-1), minlength=E)
    P = p.sum(0)
    loss = coef * E / (K * n * n) * (C * P).sum() if n else 0.0
    return dict(ids=ids, weights=w, C=C, P=P, loss=loss, s=s, p=p, z=z)


def route_grad(x, ids, dw, dloss, sigmoid=False, renorm=False, scale=1.0, coef=0.0):
    """(d_logits, a bound of the terms added up in it) for one rank's valid
    tokens; dw [n, K] or None, dloss a number."""
    n, E = x.shape
    K = ids.shape[1]
    o = route(x, K, sigmoid, renorm, scale, None, coef, ids)
    s, p, z = o["s"], o["p"], np.where(o["z"] == 0, 1.0, o["z"])
    b = dloss * coef * E / (K * n * n) * o["C"][None, :].astype(np.float64) if n else np.zeros((1, E))
    G, A = np.zeros((n, E)), np.zeros((n, E))
    if dw is not None:
        sel = np.take_along_axis(s, ids, 1)
        if renorm:
            N = sel.sum(1, keepdims=True)
            r = np.where(N == 0, 0.0, 1.0 / np.where(N == 0, 1.0, N))
            g = scale * r * (dw - (dw * sel * r).sum(1, keepdims=True))
            a = scale * r * (np.abs(dw) + (np.abs(dw) * sel * r).sum(1, keepdims=True))
        else:
            g, a = scale * dw, scale * np.abs(dw)
        np.add.at(G, (np.arange(n)[:, None], ids), g)
        np.add.at(A, (np.arange(n)[:, None], ids), a)
    if sigmoid:
        with np.errstate(over="ignore"):
            ds = s / (1.0 + np.exp(x))
        zi = np.where(o["z"] == 0, 0.0, 1.0 / z)
        d = ds * (G + (b - (p * b).sum(1, keepdims=True)) * zi)
        bound = ds * (A + (np.abs(b) + (p * np.abs(b)).sum(1, keepdims=True)) * zi)
    else:
        d = s * (G + b - (s * (G + b)).sum(1, keepdims=True))
        bound = s * (A + np.abs(b) + (s * (A + np.abs(b))).sum(1, keepdims=True))
    return d, bound


# ---- microscaling ----
def _to_grid(a, grid):
    """Index of the nearest grid value, ties to the even index, saturating."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = np.searchsorted(mid, a, side="left")
    tie = (i < len(mid)) & (a == mid[np.minimum(i, len(mid) - 1)])
    return np.where(tie & (i % 2 == 1), i + 1, i)


def _floor_log2(v):
    m, e = np.frexp(v)
    return np.where(v > 0, e - 1, -10000)


def mx_scale(x, fmt):
    """Scale byte of every 32 values of x [..., cols] (float64)."""
    amax = np.abs(x.reshape(-1, 32))
    bad = ~np.isfinite(amax).all(1)
    amax = np.where(np.isfinite(amax), amax, 0.0).max(1)
    if fmt == 4:
        e = _floor_log2(amax) - 2
    else:
        e = _floor_log2(amax) - 8
        e = np.where(amax > 448.0 * np.exp2(np.maximum(e, -300.0)), e + 1, e)
    return np.where(bad, 255, np.maximum(e, -127) + 127).astype(np.uint8).reshape(
        *x.shape[:-1], x.shape[-1] // 32)


def mx_codes(x, scale, fmt):
    """Code of every value (sign in the top bit of 4 or 8); 0 in NaN blocks."""
    grid = E2M1 if fmt == 4 else E4M3
    s = np.repeat(scale, 32, axis=-1)
    ok = s != 255
    with np.errstate(invalid="ignore"):
        a = np.where(ok, np.abs(x), 0.0) / np.exp2(s.astype(np.float64) - 127)
    i = _to_grid(a, grid)
    sign = np.signbit(x) & ok
    return (i + np.where(sign, 8 if fmt == 4 else 128, 0)).astype(np.uint8)


def mx_values(codes, scale, fmt):
    grid, top = (E2M1, 8) if fmt == 4 else (E4M3, 128)
    mag = grid[np.minimum(codes & (top - 1), len(grid) - 1)]
    s = np.repeat(scale, 32, axis=-1)
    v = np.where(codes >= top, -mag, mag) * np.exp2(s.astype(np.float64) - 127)
    return np.where(s == 255, np.nan, v)


def pack4(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack4(q):
    return np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], 2 * q.shape[-1])


def mx4(x):
    """Packed codes and scales of x."""
    s = mx_scale(x, 4)
    return pack4(mx_codes(x, s, 4)), s


def mx4_values(q, s):
    return mx_values(unpack4(q), s, 4)


# ---- the experts ----
def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def silu_slope(g):
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
        return s + g * s / (1.0 + np.exp(g))


# ---- groups ----
def plan_arrays(sizes, E, P, NvS=None):
    """A plan's arrays for group sizes [R, E+B], laid out as the planner does."""
    sizes = np.asarray(sizes, np.int64)
    padded = (sizes + P - 1) // P * P
    ends = np.cumsum(padded, 1)
    starts = ends - padded
    NvS = int(ends[:, -1].max()) if NvS is None else NvS
    assert (ends[:, -1] <= NvS).all()
    zfr = np.stack([starts + sizes, ends], 2)
    etc = np.full((sizes.shape[0], sizes.shape[1] - E), -1)
    a = dict(cu_seqlens=ends, zero_fill_ranges=zfr, experts_to_copy=etc, status=np.zeros(1))
    return {k: np.ascontiguousarray(v.astype(np.int32)) for k, v in a.items()}, NvS


def spans(arrays):
    """(rank, group, first, behind the last route, behind the padding) of groups."""
    cu, z = arrays["cu_seqlens"], arrays["zero_fill_ranges"]
    for u in range(cu.shape[0]):
        for g in range(cu.shape[1]):
            b = cu[u, g - 1] if g else 0
            if cu[u, g] > b:
                yield u, g, int(b), int(z[u, g, 0]), int(cu[u, g])


def row_kinds(arrays, NvS):
    """[R*NvS]: 1 for rows that hold routes, 2 for padding, 0 behind the groups."""
    k = np.zeros((arrays["cu_seqlens"].shape[0], NvS), np.int8)
    for u, _, a, b, c in spans(arrays):
        k[u, a:b], k[u, b:c] = 1, 2
    return k.reshape(-1)
