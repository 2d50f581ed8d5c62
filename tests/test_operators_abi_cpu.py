"""Host-side refusals of the routing and expert operators, without a GPU: each
call below is turned down before anything is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def moon():
    import combine_balanced_planning_amd as m
    return m


PTR = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4098)


def arrays(moon, **kw):
    pa = moon.moon_plan_arrays()
    pa.cu_seqlens = pa.zero_fill_ranges = pa.status = 4096
    pa.R, pa.E, pa.B, pa.NvS = 2, 8, 4, 32
    for k, v in kw.items():
        setattr(pa, k, v)
    return ctypes.byref(pa)


def config(moon, R=2, S=4, E=8, K=2, dtype=0, flags=0):
    return ctypes.byref(moon.moon_route_config(R, S, E, K, dtype, flags, 1.0, 0.0))


BAD_PLANS = [(dict(cu_seqlens=None), -1), (dict(zero_fill_ranges=4098), -1), (dict(status=None), -1),
             (dict(R=3), -2), (dict(R=0), -1), (dict(B=0), -1), (dict(NvS=0), -1), (dict(E=1024), -3),
             (dict(B=8192), -3), (dict(NvS=1 << 30), -3)]


def test_route_refusals(moon):
    def call(cfg, logits=PTR, topk=PTR, w=PTR, bias=None, loss=None, ws=None, n=0):
        return moon._lib.moon_route(cfg, logits, bias, None, topk, w, None, None, None, loss, ws, n, None)

    inv, uns = moon.MOON_ERR_INVALID_ARG, moon.MOON_ERR_UNSUPPORTED
    assert call(None) == inv
    for kw in (dict(R=0), dict(S=0), dict(E=0), dict(K=0), dict(K=9), dict(dtype=2), dict(flags=4)):
        assert call(config(moon, **kw)) == inv, kw
    for kw in (dict(R=33), dict(E=513), dict(E=512, K=65), dict(R=32, S=1 << 25, K=2)):
        assert call(config(moon, **kw)) == uns, kw
    c = config(moon)
    assert call(c, logits=None) == inv and call(c, topk=None) == inv and call(c, w=None) == inv
    assert call(c, logits=ODD) == inv and call(c, topk=ODD) == inv
    assert call(c, bias=PTR) == inv                       # a bias needs sigmoid scores
    big = config(moon, S=1000)
    n = ctypes.c_size_t(0)
    assert moon._lib.moon_route_workspace(big, ctypes.byref(n)) == 0 and n.value > 0
    assert call(big, loss=PTR) == inv                     # no workspace
    assert call(big, loss=PTR, ws=PTR, n=n.value - 1) == inv
    assert call(big, loss=PTR, ws=ODD, n=n.value) == inv
    assert moon._lib.moon_route_workspace(big, None) == inv
    assert moon._lib.moon_route_workspace(config(moon, K=9), ctypes.byref(n)) == inv


def test_route_backward_refusals(moon):
    def call(cfg, logits=PTR, topk=PTR, dw=PTR, c=PTR, n=PTR, dl=PTR, d=PTR):
        return moon._lib.moon_route_backward(cfg, logits, None, topk, dw, c, n, dl, d, None)

    inv = moon.MOON_ERR_INVALID_ARG
    cfg = config(moon)
    assert call(None) == inv and call(cfg, logits=None) == inv and call(cfg, d=None) == inv
    assert call(cfg, topk=None) == inv and call(cfg, c=None) == inv and call(cfg, n=None) == inv
    assert call(cfg, dl=ODD) == inv and call(cfg, dw=ODD) == inv
    assert call(config(moon, E=513)) == moon.MOON_ERR_UNSUPPORTED


def test_mx4_refusals(moon):
    lib, inv, uns = moon._lib, moon.MOON_ERR_INVALID_ARG, moon.MOON_ERR_UNSUPPORTED

    def quant(x=PTR, dtype=1, rows=64, cols=64, plan=None, q=PTR, s=PTR):
        return lib.moon_mx4_quantize(x, dtype, rows, cols, plan, q, s, None)

    def back(q=PTR, s=PTR, rows=64, cols=64, plan=None, dtype=1, y=PTR):
        return lib.moon_mx4_dequantize(q, s, rows, cols, plan, dtype, y, None)

    for f in (quant, back):
        for kw in (dict(q=None), dict(s=None), dict(dtype=2), dict(rows=0), dict(rows=-5), dict(cols=0),
                   dict(cols=48), dict(q=ctypes.c_void_p(4104))):
            assert f(**kw) == inv, kw
        assert f(cols=65568) == uns and f(rows=1 << 31) == uns
        assert f(plan=arrays(moon), rows=63) == inv       # not R*NvS rows
        for kw, want in BAD_PLANS:
            assert f(plan=arrays(moon, **kw)) == want, kw
    assert quant(x=None) == inv and quant(x=ctypes.c_void_p(4104)) == inv and back(y=None) == inv


def test_expert_refusals(moon):
    lib, inv, uns = moon._lib, moon.MOON_ERR_INVALID_ARG, moon.MOON_ERR_UNSUPPORTED

    def weight(**kw):
        w = moon.moon_mx4_weight(4096, 4096, 4096, 4096)
        for k, v in kw.items():
            setattr(w, k, v)
        return ctypes.byref(w)

    def gemm(plan=None, xq=PTR, xs=PTR, K=64, w=0, N=16, y=PTR):
        return lib.moon_expert_gemm_mx4(plan or arrays(moon), xq, xs, K, weight() if w == 0 else w, N, y, None)

    def swiglu(plan=None, xq=PTR, xs=PTR, K=64, w=0, N=16, y=PTR, rw=None):
        return lib.moon_expert_swiglu_mx4(plan or arrays(moon), xq, xs, K, weight(), weight() if w == 0 else w,
                                          N, rw, y, None)

    for f in (gemm, swiglu):
        for kw in (dict(xq=None), dict(xs=None), dict(y=None), dict(w=None), dict(K=0), dict(K=48),
                   dict(N=0), dict(N=12), dict(xq=ctypes.c_void_p(4104)), dict(y=ctypes.c_void_p(4104)),
                   dict(w=weight(slot_q=None)), dict(w=weight(expert_scales=None)),
                   dict(w=weight(expert_q=4104))):
            assert f(**kw) == inv, kw
        assert f(K=65568) == uns and f(N=65544) == uns
        for kw, want in BAD_PLANS:
            assert f(plan=arrays(moon, **kw)) == want, kw
    assert swiglu(rw=ODD) == inv


def test_swiglu8_refusals(moon):
    lib, inv, uns = moon._lib, moon.MOON_ERR_INVALID_ARG, moon.MOON_ERR_UNSUPPORTED

    def save(plan=None, x=PTR, w=None, F=32, h=PTR, saved=PTR, s=PTR):
        return lib.moon_swiglu_save8(plan or arrays(moon), x, w, F, h, saved, s, None)

    def grad(plan=None, x=PTR, w=None, F=32, h=PTR, saved=PTR, s=PTR, dw=None):
        return lib.moon_swiglu_grad8(plan or arrays(moon), x, saved, s, w, F, h, dw, None)

    for f in (save, grad):
        for kw in (dict(x=None), dict(h=None), dict(saved=None), dict(s=None), dict(F=0), dict(F=48),
                   dict(w=ODD), dict(x=ctypes.c_void_p(4104)), dict(h=ctypes.c_void_p(4104)),
                   dict(saved=ctypes.c_void_p(4104))):
            assert f(**kw) == inv, kw
        assert f(F=65568) == uns
        for kw, want in BAD_PLANS:
            assert f(plan=arrays(moon, **kw)) == want, kw
    assert grad(dw=ODD) == inv


def test_windows_beyond_a_launch_are_refused(moon):
    """2^29 rows a window are the most that a launch is sure to cover."""
    n = (1 << 29) + 1
    for R, status in ((1, moon.MOON_ERR_UNSUPPORTED), (2, moon.MOON_ERR_UNSUPPORTED)):
        assert moon._lib.moon_mx4_quantize(PTR, 1, R * n, 32, arrays(moon, R=R, NvS=n), PTR, PTR,
                                           None) == status
        assert moon._lib.moon_swiglu_save8(arrays(moon, R=R, NvS=n), PTR, None, 32, PTR, PTR, PTR,
                                           None) == status


def test_plan_arrays_of_no_rank_are_refused(moon):
    """A plan dict of empty arrays is an error of its arguments."""
    import torch
    i32 = dict(dtype=torch.int32)
    plan = {"cu_seqlens": torch.empty((0, 4), **i32), "experts_to_copy": torch.empty((0, 1), **i32),
            "zero_fill_ranges": torch.empty((0, 4, 2), **i32), "status": torch.empty((1,), **i32)}
    with pytest.raises(ValueError, match="cu_seqlens"):
        moon._groups(plan, 0, 0)
