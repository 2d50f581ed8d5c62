"""The routing and expert operators next to plan, dispatch and combine: their cases, plain forms and exact results.

Kinds of cases
  route       top-k routing of router logits: ids, weights and per-expert counts (serving)
  route_step  the same with the balance loss, and the gradient of both (a training step)
  weights4    expert weights to microscaled 4-bit (MXFP4) and back (loading; checking what a format costs)
  rows4       the dispatched rows of a plan to MXFP4 and back
  gemm4       MXFP4 rows times their experts' MXFP4 weights, all groups of all ranks (an expert's down projection)
  swiglu4     two such products with the gated activation (gate and up projections)
  swiglu8     gated activation that keeps its inputs in 8 bits, and its gradient from them (a training step)

`own` false: elementary torch operations in 32 bits (64 for selection keys).  `own` true: the framework's calls.
"""
import math

import numpy as np
import torch

own = False

SIGMOID, RENORM = 0x1, 0x2  # the framework's routing flags
FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decode step: a few tokens a rank behind a padded batch; latency counts
        dict(name="route decode", kind="route", R=8, E=256, K=8, S=16, score="sigmoid", renorm=True, scale=2.5, dtype="bf16", pads=True),
        # prefill of the same router
        dict(name="route prefill", kind="route", R=8, E=256, K=8, S=4096, score="sigmoid", renorm=True, scale=2.5, dtype="fp32", pads=False),
        # training at the largest configuration
        dict(name="route step r16", kind="route_step", R=16, E=384, K=8, S=8192, score="softmax", renorm=True, scale=1.0, dtype="fp32", pads=False),
        # a ragged one: odd counts, bf16 logits, weights left unnormalised
        dict(name="route step odd", kind="route_step", R=4, E=60, K=6, S=777, score="softmax", renorm=False, scale=1.0, dtype="bf16", pads=True),
        # the gate projections of 32 experts as they are loaded
        dict(name="weights to 4 bits", kind="weights4", rows=65536, cols=7168, dtype="bf16"),
        # the windows of a mid-sized layer, padding every group to 16 rows
        dict(name="rows to 4 bits", kind="rows4", R=8, E=64, K=6, S=2048, B=8, P=16, cols=2048),
        # one token a rank: bound by the weights of the experts it meets
        dict(name="swiglu decode", kind="swiglu4", R=8, E=64, K=6, S=1, B=8, P=1, cols=2048, out=1024, weighted=True),
        # a decode batch on the large model's down projection
        dict(name="gemm decode", kind="gemm4", R=8, E=256, K=8, S=16, B=4, P=16, cols=2048, out=7168),
        # prefill of the large model
        dict(name="swiglu prefill", kind="swiglu4", R=8, E=256, K=8, S=4096, B=4, P=128, cols=7168, out=2048, weighted=False),
        # the mid-sized layer's down projection
        dict(name="gemm r8-e64", kind="gemm4", R=8, E=64, K=6, S=2048, B=8, P=16, cols=1024, out=2048),
        # a training step of the large model
        dict(name="swiglu8 step", kind="swiglu8", R=8, E=256, K=8, S=4096, B=4, P=128, cols=2048, weighted=True),
        # a narrow, ragged one
        dict(name="swiglu8 odd", kind="swiglu8", R=2, E=8, K=2, S=333, B=4, P=8, cols=96, weighted=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route", "route_step", "weights4", "rows4", "gemm4", "swiglu4", "swiglu8"])
    R = rng.choice([1, 2, 4, 8, 16])
    if kind in ("route", "route_step"):
        E = R * _log_int(rng, max(1, 16 // R), 384 // R)
        return dict(kind=kind, R=R, E=E, K=rng.randint(1, min(8, E)), S=_log_int(rng, 1, 8192 * 8 // max(R, 8)), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["fp32", "bf16"]), pads=rng.random() < 0.4)
    if kind == "weights4":
        return dict(kind=kind, rows=_log_int(rng, 1, 40000), cols=32 * _log_int(rng, 1, 224), dtype=rng.choice(["fp32", "bf16"]))
    Eg = _log_int(rng, 1, 256 // R)
    K = rng.randint(1, min(8, R * Eg))
    P = rng.choice([1, 8, 16, 128])
    S = _log_int(rng, 1, 16384 // (R * K))
    c = dict(kind=kind, R=R, E=R * Eg, K=K, S=S, B=rng.randint(1, min(8, Eg)), P=P)
    if kind == "rows4":
        return dict(c, cols=32 * _log_int(rng, 1, 224))
    if kind == "swiglu8":
        return dict(c, cols=32 * _log_int(rng, 1, 64), weighted=rng.random() < 0.5)
    cols = 32 * _log_int(rng, 2, 224)
    if kind == "gemm4":
        return dict(c, cols=cols, out=8 * _log_int(rng, 4, 512))
    return dict(c, cols=cols, out=32 * _log_int(rng, 1, 64), weighted=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs
def _nvs(c):
    P, Eg = c["P"], c["E"] // c["R"]
    return (c["S"] * c["K"] + (Eg + c["B"]) * (P - 1) + P - 1) // P * P


def _sizes(c, seed):
    """Rows of every group, [R, E+B]: each rank holds exactly S*K, spread unevenly over its own experts and a few slots."""
    rng = np.random.default_rng(seed)
    R, E, B, N = c["R"], c["E"], c["B"], c["S"] * c["K"]
    Eg = E // R
    n = np.zeros((R, E + B), np.int64)
    for u in range(R):
        p = np.exp(0.5 * rng.standard_normal(Eg + B))
        used = int(rng.integers(0, min(B, Eg) + 1)) if R > 1 else 0
        p[Eg:Eg + used] *= 0.5
        p[Eg + used:] = 0
        m = rng.multinomial(N, p / p.sum())
        n[u, u * Eg:(u + 1) * Eg] = m[:Eg]
        n[u, E:] = m[Eg:]
    return n


def _plan(c, seed):
    """A plan's arrays of these sizes, as the planner lays them out, and the rows of the largest group."""
    n = _sizes(c, seed)
    R, E, B, P = c["R"], c["E"], c["B"], c["P"]
    Eg = E // R
    ends = np.cumsum((n + P - 1) // P * P, axis=1)
    starts = ends - (n + P - 1) // P * P
    zfr = np.stack([starts + n, ends], axis=2)
    etc = np.full((R, B), -1, np.int64)
    for u in range(R):
        donor = (u + 1) % R
        used = np.flatnonzero(n[u, E:] > 0)
        etc[u, used] = donor * Eg + used
    nvs = _nvs(c)
    rng = np.random.default_rng(seed + 1)
    rows = np.concatenate([u * nvs + np.concatenate([np.arange(s, s + k) for s, k in zip(starts[u], n[u])]) for u in range(R)])
    dst = rng.permutation(rows).reshape(R, -1)
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a.astype(np.int32))).cuda()  # noqa: E731
    return dict(dst=put(dst), experts_to_copy=put(etc), zero_fill_ranges=put(zfr), cu_seqlens=put(ends), status=torch.zeros(1, dtype=torch.int32, device="cuda")), int(n.max())


def _real(c, plan):
    """The rows that hold routes, [R*NvS] of 0 and 1."""
    return _places(c, plan)[1]


def _normal(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _codes(shape, g):
    """Packed 4-bit values as a bell curve leaves them after scaling by its block's largest value."""
    p = np.exp(-0.5 * (np.array(FP4) / 1.9) ** 2) * np.array([0.5, 0.5, 0.5, 0.5, 0.75, 1, 1.5, 1.5])
    t = np.repeat(np.arange(8), np.maximum(1, np.round(128 * p / p.sum()).astype(int)))[:128]
    t = np.concatenate([t, np.zeros(128 - len(t), int)])
    t = torch.from_numpy(np.concatenate([t, t + 8]).astype(np.uint8)).cuda()
    out = torch.empty(shape, dtype=torch.uint8, device="cuda").view(-1)
    for a in range(0, out.numel(), 1 << 28):
        n = min(1 << 28, out.numel() - a)
        lo, hi = (t[torch.randint(0, 256, (n,), generator=g, device="cuda", dtype=torch.uint8).int()] for _ in range(2))
        out[a:a + n] = lo | (hi << 4)
    return out.view(shape)


def _scales(shape, g, mid):
    return torch.randint(mid - 2, mid + 2, shape, generator=g, device="cuda", dtype=torch.uint8)


def prepare(case, seed):
    c, g = dict(case), torch.Generator("cuda").manual_seed(seed)
    kind = c["kind"]
    dt = {"fp32": torch.float32, "bf16": torch.bfloat16}[c.get("dtype", "bf16")]
    if kind in ("route", "route_step"):
        R, S, E, K = c["R"], c["S"], c["E"], c["K"]
        s = dict(case=c)
        skew = -0.5 * torch.log1p(torch.randperm(E, generator=g, device="cuda").float())
        s["logits"] = (_normal((R, S, E), g) + skew).to(dt)
        s["bias"] = 0.05 * _normal((E,), g) if c["score"] == "sigmoid" else None
        s["valid"] = torch.arange(S, device="cuda") < torch.randint(1, S + 1, (R, 1), generator=g, device="cuda") if c["pads"] else None
        s["topk"] = torch.zeros((R, S, K), dtype=torch.int32, device="cuda")
        s["weights"] = torch.zeros((R, S, K), device="cuda")
        s["counts"] = torch.zeros((R, E), dtype=torch.int32, device="cuda")
        if kind == "route_step":
            s["tokens"] = torch.zeros((R,), dtype=torch.int32, device="cuda")
            s["prob_sums"] = torch.zeros((R, E), device="cuda")
            s["loss"] = torch.zeros((R,), device="cuda")
            s["d_weights"] = _normal((R, S, K), g)
            s["d_loss"] = torch.full((R,), float(S), device="cuda")
            s["d_logits"] = torch.zeros((R, S, E), dtype=dt, device="cuda")
        return s
    if kind == "weights4":
        n, w = c["rows"], c["cols"]
        s = dict(case=c, x=_normal((n, w), g).mul_(w ** -0.5).to(dt))
        return dict(s, q=torch.zeros((n, w // 2), dtype=torch.uint8, device="cuda"), scales=torch.zeros((n, w // 32), dtype=torch.uint8, device="cuda"), y=torch.zeros((n, w), dtype=dt, device="cuda"))
    plan, cap = _plan(c, seed)
    rows, w, R = c["R"] * _nvs(c), c["cols"], c["R"]
    s = dict(case=c, plan=plan, cap=cap)
    real = _real(c, plan)
    if kind == "rows4":
        s["x"] = (_normal((rows, w), g) * real[:, None]).bfloat16()
        s["q"] = torch.zeros((rows, w // 2), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros((rows, w // 32), dtype=torch.uint8, device="cuda")
        s["y"] = torch.zeros((rows, w), dtype=torch.bfloat16, device="cuda")
        return s
    if kind == "swiglu8":
        s["x"] = (_normal((rows, 2 * w), g) * real[:, None]).bfloat16()
        s["dh"] = (_normal((rows, w), g) * real[:, None]).bfloat16()
        s["weights"] = torch.rand((rows,), generator=g, device="cuda") * real if c["weighted"] else None
        s["d_weights"] = torch.zeros((rows,), device="cuda") if c["weighted"] else None
        s["saved"] = torch.zeros((rows, 2 * w), dtype=torch.uint8, device="cuda")
        s["saved_scales"] = torch.zeros((rows, w // 16), dtype=torch.uint8, device="cuda")
        s["h"] = torch.zeros((rows, w), dtype=torch.bfloat16, device="cuda")
        s["dx"] = torch.zeros((rows, 2 * w), dtype=torch.bfloat16, device="cuda")
        return s
    n = c["out"]
    s["xq"], s["xs"] = _codes((rows, w // 2), g), _scales((rows, w // 32), g, 126)
    mid = 126 - int(round(0.5 * math.log2(w)))  # weights of about 1/sqrt(cols)
    s["w"] = []
    for _ in range(2 if kind == "swiglu4" else 1):
        e, es = _codes((c["E"], n, w // 2), g), _scales((c["E"], n, w // 32), g, mid)
        i = plan["experts_to_copy"].long().clamp(min=0)
        s["w"].append((e, es, e[i], es[i]))
    s["weights"] = torch.rand((rows,), generator=g, device="cuda") * real if c.get("weighted") else None
    s["y"] = torch.zeros((rows, n), dtype=torch.bfloat16, device="cuda")
    return s


# ---------------------------------------------------------------- the operators
def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import combine_balanced_planning_amd as moon
    c = s["case"]
    kind = c["kind"]
    if kind in ("route", "route_step"):
        flags = (moon.MOON_ROUTE_SIGMOID if c["score"] == "sigmoid" else 0) | (moon.MOON_ROUTE_RENORM if c["renorm"] else 0)
        if kind == "route":
            moon.moon_route(s["logits"], s["topk"], s["weights"], flags, c["scale"], bias=s["bias"], valid=s["valid"], tokens_per_expert=s["counts"])
            return dict(topk=s["topk"], weights=s["weights"], counts=s["counts"])
        moon.moon_route(s["logits"], s["topk"], s["weights"], flags, c["scale"], bias=s["bias"], valid=s["valid"], tokens_per_expert=s["counts"],
                        valid_tokens=s["tokens"], prob_sums=s["prob_sums"], loss=s["loss"], loss_coef=0.01)
        moon.moon_route_backward(s["logits"], s["topk"], s["d_logits"], flags, c["scale"], valid=s["valid"], d_weights=s["d_weights"],
                                 tokens_per_expert=s["counts"], valid_tokens=s["tokens"], d_loss=s["d_loss"], loss_coef=0.01)
        return dict(topk=s["topk"], weights=s["weights"], counts=s["counts"], prob_sums=s["prob_sums"], loss=s["loss"], d_logits=s["d_logits"])
    if kind in ("weights4", "rows4"):
        moon.moon_mx4_quantize(s["x"], s["q"], s["scales"], plan=s.get("plan"))
        moon.moon_mx4_dequantize(s["q"], s["scales"], s["y"], plan=s.get("plan"))
        return s["y"]
    if kind == "gemm4":
        moon.moon_expert_gemm_mx4(s["plan"], s["xq"], s["xs"], s["w"][0], s["y"])
        return s["y"]
    if kind == "swiglu4":
        moon.moon_expert_swiglu_mx4(s["plan"], s["xq"], s["xs"], s["w"][0], s["w"][1], s["y"], row_weights=s["weights"])
        return s["y"]
    moon.moon_swiglu_save8(s["plan"], s["x"], s["h"], s["saved"], s["saved_scales"], row_weights=s["weights"])
    moon.moon_swiglu_grad8(s["plan"], s["dh"], s["saved"], s["saved_scales"], s["dx"], row_weights=s["weights"], d_row_weights=s["d_weights"])
    return [s["h"], s["dx"], s["d_weights"]]


def _plain(s):
    kind = s["case"]["kind"]
    if kind in ("route", "route_step"):
        return _plain_route(s)
    if kind in ("weights4", "rows4"):
        y = _fp4(s["x"].float())
        return (y if kind == "weights4" else y * _real(s["case"], s["plan"])[:, None]).to(s["x"].dtype)
    return _plain_swiglu8(s) if kind == "swiglu8" else _plain_product(s)


def _plain_route(s):
    c, x = s["case"], s["logits"].float()
    R, S, E = x.shape
    K, sig = c["K"], c["score"] == "sigmoid"
    key = torch.sigmoid(x.double()) + s["bias"].double() if sig else x
    top = torch.sort(key, dim=-1, descending=True, stable=True)[1][..., :K]
    p = torch.sigmoid(x) if sig else torch.softmax(x, -1)
    total = p.sum(-1, keepdim=True)
    prob = p / total
    sel = p.gather(-1, top)
    norm = sel.sum(-1, keepdim=True) if c["renorm"] else torch.ones_like(sel[..., :1])
    w = c["scale"] * sel / norm
    ok = torch.ones((R, S), dtype=torch.bool, device=x.device) if s["valid"] is None else s["valid"]
    topk = torch.where(ok[..., None], top, 0).int()
    w = torch.where(ok[..., None], w, 0.0)
    counts = torch.zeros((R, E), dtype=torch.int32, device=x.device).scatter_add_(1, topk.view(R, -1).long(), torch.ones((R, S * K), dtype=torch.int32, device=x.device))
    out = dict(topk=topk, weights=w, counts=counts)
    if c["kind"] == "route":
        return out
    n = ok.sum(1).float()
    real = counts.clone()
    real[:, 0] -= (K * (S - ok.sum(1))).int()
    sums = torch.where(ok[..., None], prob, 0.0).sum(1)
    b = 0.01 * E / (K * n[:, None] ** 2) * real
    out["prob_sums"], out["loss"] = sums, (b * sums).sum(1)
    b = (b * s["d_loss"][:, None])[:, None, :].expand(R, S, E)
    dw = s["d_weights"]
    gs = c["scale"] / norm * (dw - (dw * sel / norm).sum(-1, keepdim=True) if c["renorm"] else dw)
    gk = torch.zeros_like(x).scatter_(-1, top, gs)
    if sig:
        d = (gk + (b - (b * prob).sum(-1, keepdim=True)) / total) * p * torch.sigmoid(-x)
    else:
        d = p * (gk + b - (p * (gk + b)).sum(-1, keepdim=True))
    out["d_logits"] = torch.where(ok[..., None], d, 0.0).to(s["logits"].dtype)
    return out


def _fp4(x):
    """Each 32 values of the last axis on the 4-bit grid under their power-of-two scale."""
    v = x.view(*x.shape[:-1], -1, 32)
    e = (torch.frexp(v.abs().amax(-1, keepdim=True))[1] - 3).clamp(min=-127)
    a = torch.ldexp(v.abs(), -e)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0)
    return torch.ldexp(torch.copysign(q, v), e).view(x.shape)


def _fp8(x):
    """Each 32 values of the last axis as e4m3 under the smallest power-of-two scale that holds them."""
    v = x.view(*x.shape[:-1], -1, 32)
    m, e = torch.frexp(v.abs().amax(-1, keepdim=True))
    e = (e - torch.where(m > 0.875, 8, 9)).clamp(min=-127)
    return torch.ldexp(torch.ldexp(v, -e).to(torch.float8_e4m3fn).float(), e).view(x.shape)


def _places(c, plan):
    """For every window row: its group (rank by rank, a rank's own experts and then its slots), whether a route is there, and its place in the group."""
    R, E, B = c["R"], c["E"], c["B"]
    Eg, nvs = E // R, _nvs(c)
    cu, zfr = plan["cu_seqlens"], plan["zero_fill_ranges"]
    r = torch.arange(nvs, device=cu.device, dtype=torch.int32).expand(R, nvs).contiguous()
    g = torch.searchsorted(cu, r, right=True)
    inside = g < E + B
    g = g.clamp(max=E + B - 1)
    start = torch.where(g > 0, cu.gather(1, (g - 1).clamp(min=0)), 0)
    real = inside & (r < zfr[..., 0].gather(1, g))
    u = torch.arange(R, device=cu.device)[:, None]
    entry = u * (Eg + B) + torch.where(g < E, (g - u * Eg).clamp(0, Eg - 1), Eg + g - E)
    return entry.view(-1), real.view(-1), (r - start).view(-1)


def _values4(q, s):
    """The numbers of packed 4-bit values and their scales."""
    t = torch.tensor(FP4 + tuple(-v for v in FP4), device=q.device)
    v = torch.stack([t[(q & 15).int()], t[(q >> 4).int()]], -1).flatten(-2)
    return (v.view(*v.shape[:-1], -1, 32) * torch.exp2(s.float() - 127).unsqueeze(-1)).view(v.shape)


def _plain_product(s):
    c, cap = s["case"], s["cap"]
    R, E, B = c["R"], c["E"], c["B"]
    Eg, n = E // R, c["out"]
    groups = R * (Eg + B)
    entry, real, pos = _places(c, s["plan"])
    x = _values4(s["xq"], s["xs"])
    at = torch.where(real, entry * cap + pos, groups * cap)
    xp = torch.zeros((groups * cap + 1, x.shape[1]), device=x.device).index_copy_(0, at, x)[:-1].view(groups, cap, -1)
    ys = []
    for e, es, sl, ss in s["w"]:
        q = torch.cat([e.view(R, Eg, n, -1), sl], 1).view(groups, n, -1)
        w = _values4(q, torch.cat([es.view(R, Eg, n, -1), ss], 1).view(groups, n, -1))
        ys.append(torch.bmm(xp, w.transpose(1, 2)).view(groups * cap, n)[at.clamp(max=groups * cap - 1)])
        del w, q
    y = ys[0] if len(ys) == 1 else ys[0] * torch.sigmoid(ys[0]) * ys[1]
    if s["weights"] is not None:
        y = y * s["weights"][:, None]
    return torch.where(real[:, None], y, 0.0).bfloat16()


def _plain_swiglu8(s):
    w, real = s["weights"], _real(s["case"], s["plan"])[:, None]
    gate, up = s["x"].float().chunk(2, -1)
    rw = 1.0 if w is None else w[:, None]
    h = torch.where(real, rw * (gate * torch.sigmoid(gate) * up), 0.0).bfloat16()
    gate, up = _fp8(s["x"].float()).chunk(2, -1)
    dh, sg = s["dh"].float(), torch.sigmoid(gate)
    act = gate * sg
    dx = torch.cat([dh * rw * up * sg * (1 + gate * (1 - sg)), dh * rw * act], -1)
    dx = torch.where(real, dx, 0.0).bfloat16()
    return [h, dx, None if w is None else torch.where(real[:, 0], (dh * act * up).sum(-1), 0.0)]


# ---------------------------------------------------------------- work
def work(case):
    c = case
    kind = c["kind"]
    if kind in ("route", "route_step"):
        tok, E, K = c["R"] * c["S"], c["E"], c["K"]
        b = 4 if c["dtype"] == "fp32" else 2
        move = tok * (E * b + 8 * K) + 4 * c["R"] * E
        flops = tok * (5 * E + E + 4 * K)  # exponentials and sums, one comparison each, the weights
        if kind == "route_step":
            move += tok * (E * b + 4 * K) + 8 * c["R"] * E  # d_weights read and d_logits written; the logits count once
            flops += tok * 10 * E
        return {"bytes": move, "flops": flops}
    if kind == "weights4":
        b, n = (4 if c["dtype"] == "fp32" else 2), c["rows"] * c["cols"]
        return {"bytes": 2 * n * b + n * 17 // 16, "flops": 6 * n}  # the 4-bit values and their scales written and read
    rows = c["R"] * c["S"] * c["K"]
    if kind == "rows4":
        return {"bytes": rows * c["cols"] * 81 // 16, "flops": 6 * rows * c["cols"]}
    if kind == "swiglu8":
        extra = 8 * rows if c["weighted"] else 0
        return {"bytes": rows * c["cols"] * 129 // 8 + extra, "flops": 30 * rows * c["cols"]}  # inputs, outputs, the saved bytes and scales written and read
    p, n, w = (2 if kind == "swiglu4" else 1), c["out"], c["cols"]
    met = round(sum(np.count_nonzero(_sizes(c, k)) for k in range(4)) / 4)  # groups that hold rows: each reads its expert
    return {"bytes": (rows * w + p * met * n * w) * 17 // 32 + rows * n * 2, "flops": 2 * p * rows * n * w}


# ---------------------------------------------------------------- exact results
def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("route", "route_step"):
        return _exact_route(s)
    if kind in ("weights4", "rows4"):
        y = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        for a in range(0, y.shape[0], 8192):
            y[a:a + 8192] = _nearest(s["x"][a:a + 8192].double(), FP4, 2, False)
        if kind == "rows4":
            y[~_row_mask(s)] = 0
        return y
    return _exact_swiglu8(s) if kind == "swiglu8" else _exact_product(s)


def _exact_route(s):
    c = s["case"]
    R, S, E, K = c["R"], c["S"], c["E"], c["K"]
    outs = []
    for r in range(R):  # rank by rank
        n = S if s["valid"] is None else int(s["valid"][r].sum())
        x = s["logits"][r, :n].double()
        score = 1 / (1 + torch.exp(-x)) if c["score"] == "sigmoid" else torch.exp(x - x.max(1, keepdim=True)[0])
        if c["score"] == "softmax":
            score = score / score.sum(1, keepdim=True)
        key = (score + s["bias"].double() if s["bias"] is not None else x).clone()
        ids = []
        for _ in range(K):  # the largest key that is left; the lowest id among equals
            big = key.max(1, keepdim=True)[0]
            i = torch.where(key == big, torch.arange(E, device="cuda"), E).min(1, keepdim=True)[0]
            ids.append(i)
            key.scatter_(1, i, -math.inf)
        ids = torch.cat(ids, 1)
        picked = score.gather(1, ids)
        den = picked.sum(1, keepdim=True) if c["renorm"] else torch.ones_like(picked[:, :1])
        pad = lambda t, fill: torch.cat([t, torch.full((S - n, *t.shape[1:]), fill, dtype=t.dtype, device="cuda")])  # noqa: E731
        o = dict(topk=pad(ids, 0).int(), weights=pad(c["scale"] * picked / den, 0.0))
        load = torch.bincount(ids.flatten(), minlength=E)
        o["counts"] = load.int()
        o["counts"][0] += K * (S - n)
        if c["kind"] == "route_step":
            z = score.sum(1, keepdim=True)
            o["prob_sums"] = (score / z).sum(0)
            coef = 0.01 * E * load.double() / (K * float(n) ** 2)
            o["loss"] = (coef * o["prob_sums"]).sum()
            coef = coef * s["d_loss"][r].double()
            dw = s["d_weights"][r, :n].double()
            # the score's gradient: of the weights at the picked ids, of the loss through score / sum of scores everywhere
            dpick = c["scale"] * dw / den
            if c["renorm"]:
                dpick = dpick - c["scale"] * (dw * picked).sum(1, keepdim=True) / den ** 2
            ds = (coef - (score @ coef)[:, None] / z) / z
            ds.scatter_add_(1, ids, dpick)
            dx = ds * score * (1 / (1 + torch.exp(x))) if c["score"] == "sigmoid" else score * (ds - (ds * score).sum(1, keepdim=True))
            o["d_logits"] = pad(dx, 0.0)
        outs.append(o)
    return {k: torch.stack([o[k] for o in outs]) for k in outs[0]}


def _nearest(x, grid, top_exponent, hold):
    """x on the signed `grid` under the power-of-two scale of each 32 values, ties to the even place of the grid; `hold`: no value may pass the grid's end."""
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    v = x.reshape(-1, 32)
    big = v.abs().amax(1, keepdim=True)
    e = torch.where(big > 0, torch.floor(torch.log2(big.clamp(min=1e-60))), -1000.0)
    e = torch.where(torch.exp2(e) > big, e - 1, e)  # log2 rounds
    e = torch.where((torch.exp2(e + 1) <= big) & (big > 0), e + 1, e)
    e = e - top_exponent
    if hold:
        e = torch.where(big > grid[-1] * torch.exp2(e), e + 1, e)
    scale = torch.exp2(e.clamp(min=-127))
    a = v.abs() / scale
    mid = (grid[1:] + grid[:-1]) / 2
    i = torch.searchsorted(mid, a.contiguous())  # midpoints below a
    at_mid = (i < len(mid)) & (mid[i.clamp(max=len(mid) - 1)] == a)
    i = torch.where(at_mid & (i % 2 == 1), i + 1, i)
    return (torch.sign(v) * grid[i] * scale).view(x.shape)


def _row_mask(s):
    m = torch.zeros((s["case"]["R"], _nvs(s["case"])), dtype=torch.bool, device="cuda")
    for u, _, a, b in _groups(s):
        m[u, a:b] = True
    return m.view(-1)


def _groups(s):
    """(rank, group, first row, row behind the last) of every group that holds rows."""
    cu, z = s["plan"]["cu_seqlens"].cpu().numpy(), s["plan"]["zero_fill_ranges"].cpu().numpy()
    return [(u, j, int(cu[u, j - 1]) if j else 0, int(z[u, j, 0])) for u in range(cu.shape[0]) for j in range(cu.shape[1]) if z[u, j, 0] > (cu[u, j - 1] if j else 0)]


def _exact_swiglu8(s):
    grid = [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** k for k in range(-6, 9) for m in range(8) if not (k == 8 and m == 7)]
    f, mask = s["case"]["cols"], _row_mask(s)
    h, dx = (torch.zeros(s[k].shape, dtype=torch.float64, device="cuda") for k in ("h", "dx"))
    dw = None if s["weights"] is None else torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
    for a in range(0, h.shape[0], 16384):
        b = slice(a, a + 16384)
        x, dh = s["x"][b].double(), s["dh"][b].double()
        rw = mask[b, None].double() if dw is None else s["weights"][b, None].double()
        h[b] = rw * x[:, :f] / (1 + torch.exp(-x[:, :f])) * x[:, f:]
        x = _nearest(x, grid, 8, True)
        t = 1 / (1 + torch.exp(-x[:, :f]))
        dx[b, :f] = rw * dh * x[:, f:] * (t + x[:, :f] * t * (1 - t))
        dx[b, f:] = rw * dh * x[:, :f] * t
        if dw is not None:
            dw[b] = mask[b] * (dh * x[:, :f] * t * x[:, f:]).sum(1)
    return [h, dx, dw]


def _exact_product(s):
    c = s["case"]
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda").view(c["R"], -1, c["out"])
    grid = np.array(FP4 + tuple(-v for v in FP4))
    pair = torch.from_numpy(np.stack([grid[np.arange(256) % 16], grid[np.arange(256) // 16]], 1)).cuda()

    def number(q, sc):
        v = pair[q.long()].reshape(*q.shape[:-1], -1, 32)
        return (v * torch.pow(2.0, sc.double() - 127)[..., None]).flatten(-2)

    xq, xs = (s[k].view(c["R"], -1, s[k].shape[1]) for k in ("xq", "xs"))
    for u, j, a, b in _groups(s):
        x = number(xq[u, a:b], xs[u, a:b])
        p = [x @ number(*((e[j], es[j]) if j < c["E"] else (sl[u, j - c["E"]], ss[u, j - c["E"]]))).T for e, es, sl, ss in s["w"]]
        v = p[0] if len(p) == 1 else p[0] / (1 + torch.exp(-p[0])) * p[1]
        y[u, a:b] = v if s["weights"] is None else v * s["weights"].view(c["R"], -1)[u, a:b, None].double()
    return y.view(s["y"].shape)
