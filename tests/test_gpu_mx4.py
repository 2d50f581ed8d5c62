"""GPU parity of the MXFP4 conversions: codes, scales and values read back are
compared bit for bit with the 64-bit reference (power-of-two scales leave one
rounding, so nothing may differ)."""
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


def same(a, b):
    return np.array_equal(a, b, equal_nan=True)


def round_trip(env, x, plan=None, fill=0xEE):
    moon, torch, dev = env
    rows, cols = x.shape
    q = torch.full((rows, cols // 2), fill, dtype=torch.uint8, device=dev)
    s = torch.full((rows, cols // 32), fill, dtype=torch.uint8, device=dev)
    y = torch.full((rows, cols), 77.0, dtype=x.dtype, device=dev)
    moon.moon_mx4_quantize(x, q, s, plan=plan)
    moon.moon_mx4_dequantize(q, s, y, plan=plan)
    torch.cuda.synchronize()
    return q.cpu().numpy(), s.cpu().numpy(), y.double().cpu().numpy()


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (5, 96), (1, 2048), (7, 544), (257, 32),
                                       (33, 4096), (4200, 160), (2, 65536)])
def test_round_trip(env, rows, cols, bf16):
    say(f"[case] mx4 {rows}x{cols} bf16={bf16}")
    moon, torch, dev = env
    rng = np.random.default_rng(rows * 7 + cols)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-30, 30, (rows, cols // 32)).repeat(32, 1))
    x = torch.from_numpy(x.astype(np.float32)).to(dev)
    x = x.bfloat16() if bf16 else x
    q, s, y = round_trip(env, x)
    wq, ws = ref.mx4(x.double().cpu().numpy())
    assert (s == ws).all()
    assert (q == wq).all()
    assert same(y, ref.mx4_values(wq, ws))


def test_every_bf16_pattern(env):
    """All 65536 bit patterns, each under the block scales that a neighbour of
    every binade gives it: rounding, ties, saturation, subnormals, NaN."""
    moon, torch, dev = env
    bits = np.arange(65536, dtype=np.uint16)
    for lift in (0, 1, 2, 3, 4, 7):
        say(f"[case] all bf16 patterns, neighbour {lift} binades up")
        x = np.zeros((65536, 32), np.uint16)
        x[:, 5] = bits
        up = np.minimum((bits & 0x7FFF) + (lift << 7), 0x7F7F).astype(np.uint16)
        x[:, 20] = np.where((bits & 0x7F80) == 0x7F80, 0, up)
        t = torch.from_numpy(x.view(np.int16)).to(dev).view(torch.bfloat16)
        v = t.double().cpu().numpy()
        q, s, y = round_trip(env, t)
        wq, ws = ref.mx4(v)
        assert (s == ws).all()
        assert (q == wq).all()
        assert same(y, ref.mx4_values(wq, ws))


def test_fp32_extremes(env):
    moon, torch, dev = env
    say("[case] fp32 extremes")
    v = np.array([0.0, -0.0, 1e-45, -1e-45, 1.1754944e-38, 5e-39, 3.4028235e38, -3.4028235e38, np.inf,
                  -np.inf, np.nan, 1.0, 0.24999999, 0.25, 0.25000003, 5.0, 4.9999995, 5.0000005, 7.9999995,
                  6.0, 3.5, 2.5, 1.75, 1.25, 0.75, 2.0 ** -126, 2.0 ** -127, 2.0 ** -128], np.float32)
    x = np.zeros((2 * len(v), 32), np.float32)
    x[:len(v), 0] = v
    x[len(v):, 31] = v
    x[len(v):, 3] = 4.0
    q, s, y = round_trip(env, torch.from_numpy(x).to(dev))
    wq, ws = ref.mx4(x.astype(np.float64))
    assert (s == ws).all() and (q == wq).all() and same(y, ref.mx4_values(wq, ws))


def test_every_code_and_scale_reads_back(env):
    """All 16 codes under all 256 scales, to fp32 and bf16: exact but for what
    bf16 or fp32 cannot hold (beyond its largest finite: infinity)."""
    moon, torch, dev = env
    q = np.tile(ref.pack4(np.arange(32, dtype=np.uint8) % 16), (256, 1))
    s = np.arange(256, dtype=np.uint8)[:, None]
    want = ref.mx4_values(q, s)
    for dt in (torch.float32, torch.bfloat16):
        y = torch.empty((256, 32), dtype=dt, device=dev)
        moon.moon_mx4_dequantize(torch.from_numpy(q).to(dev), torch.from_numpy(s).to(dev), y)
        w = torch.from_numpy(want).to(dt).double().numpy()
        assert same(y.double().cpu().numpy(), w)


SIZES = [
    # E, P, group sizes per rank (own experts of all ranks, then slots)
    (2, 1, [[0, 5, 1], [0, 0, 0]][:1]),
    (4, 8, [[3, 0, 0, 0, 9, 0], [0, 0, 1, 16, 0, 0]]),
    (2, 128, [[1, 0, 129, 0], [0, 64, 0, 127]]),
    (6, 5, [[70, 0, 0, 0, 0, 0, 3, 0], [0, 0, 1, 1, 0, 0, 0, 0], [0, 0, 0, 0, 0, 2, 64, 65]]),
]


@pytest.mark.parametrize("i", range(len(SIZES)))
@pytest.mark.parametrize("cols", [32, 224, 2048])
def test_planned_rows(env, i, cols):
    """Rows that hold routes are converted, padding (NaN here) is zeroed, rows
    behind the groups keep what they held; a failed plan writes nothing."""
    moon, torch, dev = env
    E, P, sizes = SIZES[i]
    if len(sizes) == 1:
        E = 2
    arrays, NvS = ref.plan_arrays(sizes, E, P)
    NvS += 9
    say(f"[case] planned rows {i} cols={cols} NvS={NvS}")
    R = len(sizes)
    rng = np.random.default_rng(i)
    x = rng.standard_normal((R * NvS, cols)).astype(np.float32)
    kind = ref.row_kinds(arrays, NvS)
    x[kind != 1] = np.nan
    plan = {k: torch.from_numpy(v).to(dev) for k, v in arrays.items()}
    for bf16 in (False, True):
        t = torch.from_numpy(x).to(dev)
        t = t.bfloat16() if bf16 else t
        q, s, y = round_trip(env, t, plan)
        wq, ws = ref.mx4(t.double().cpu().numpy()[kind == 1])
        assert (q[kind == 1] == wq).all() and (s[kind == 1] == ws).all()
        assert same(y[kind == 1], ref.mx4_values(wq, ws))
        assert (q[kind == 2] == 0).all() and (s[kind == 2] == 0).all() and (y[kind == 2] == 0).all()
        assert (q[kind == 0] == 0xEE).all() and (s[kind == 0] == 0xEE).all()
        assert (y[kind == 0] == 77).all()
    plan["status"].fill_(1)
    q, s, y = round_trip(env, torch.from_numpy(x).to(dev), plan)
    assert (q == 0xEE).all() and (s == 0xEE).all() and (y == 77).all()


@pytest.mark.parametrize("planned", [False, True])
def test_rows_beyond_32_bit_offsets(env, planned):
    """2.4e9 values (4.8 GB of bf16): rows at both ends."""
    moon, torch, dev = env
    rows, cols = 300000, 8192
    plan = None
    if planned:
        arrays, rows = ref.plan_arrays([[rows, 0]], 1, 1)
        plan = {k: torch.from_numpy(v).to(dev) for k, v in arrays.items()}
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev).normal_(generator=torch.Generator(device=dev).manual_seed(2))
    q = torch.zeros((rows, cols // 2), dtype=torch.uint8, device=dev)
    s = torch.zeros((rows, cols // 32), dtype=torch.uint8, device=dev)
    y = torch.zeros_like(x)
    moon.moon_mx4_quantize(x, q, s, plan=plan)
    moon.moon_mx4_dequantize(q, s, y, plan=plan)
    for at in (slice(0, 3), slice(rows - 5, rows)):
        wq, ws = ref.mx4(x[at].double().cpu().numpy())
        assert (q[at].cpu().numpy() == wq).all() and (s[at].cpu().numpy() == ws).all()
        assert same(y[at].double().cpu().numpy(), ref.mx4_values(wq, ws))


def test_scales_off_their_words(env):
    """Scale bytes may start anywhere; rows of 128 values and more store them
    four at a time only where they lie on whole words."""
    moon, torch, dev = env
    x = torch.randn((37, 256), device=dev).bfloat16()
    q = torch.zeros((37, 128), dtype=torch.uint8, device=dev)
    wq, ws = ref.mx4(x.double().cpu().numpy())
    for off in (1, 2, 3, 4):
        buf = torch.full((37 * 8 + 8,), 0xEE, dtype=torch.uint8, device=dev)
        s = buf[off:off + 37 * 8].view(37, 8)
        moon.moon_mx4_quantize(x, q, s)
        assert (s.cpu().numpy() == ws).all() and (q.cpu().numpy() == wq).all()
        assert (buf[:off] == 0xEE).all() and (buf[off + 37 * 8:] == 0xEE).all()


def test_weights_of_three_axes_and_graph(env):
    """[E, N, K] weights in one call; captured and replayed on new values."""
    moon, torch, dev = env
    g = torch.Generator(device=dev).manual_seed(1)
    sets = [torch.randn((3, 40, 96), generator=g, device=dev).bfloat16() for _ in range(3)]
    x, side = sets[0].clone(), torch.cuda.Stream(device=dev)
    q = torch.zeros((3, 40, 48), dtype=torch.uint8, device=dev)
    s = torch.zeros((3, 40, 3), dtype=torch.uint8, device=dev)
    y = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moon.moon_mx4_quantize(x, q, s)
        moon.moon_mx4_dequantize(q, s, y)
    for i in (1, 2, 0, 2):
        x.copy_(sets[i])
        graph.replay()
        torch.cuda.synchronize()
        wq, ws = ref.mx4(sets[i].double().cpu().numpy())
        assert (q.cpu().numpy() == wq).all() and (s.cpu().numpy() == ws).all()
        assert same(y.double().cpu().numpy(), ref.mx4_values(wq, ws))
        x.mul_(2)
    side.wait_stream(torch.cuda.current_stream())
    q.zero_()
    side.wait_stream(torch.cuda.current_stream())
    moon.moon_mx4_quantize(sets[1], q, s, stream=side)
    side.synchronize()
    assert (q.cpu().numpy() == ref.mx4(sets[1].double().cpu().numpy())[0]).all()


def test_refusals(env):
    moon, torch, dev = env
    u8 = lambda *n: torch.zeros(n, dtype=torch.uint8, device=dev)  # noqa: E731
    x = torch.zeros((4, 64), device=dev)
    for a in (dict(x=x.half()), dict(q=u8(4, 31)), dict(scales=u8(4, 3)), dict(q=u8(4, 32).int()),
              dict(x=x.cpu()), dict(x=x.t()), dict(x=x[0])):
        k = dict(x=x, q=u8(4, 32), scales=u8(4, 2))
        k.update(a)
        with pytest.raises(ValueError):
            moon.moon_mx4_quantize(**k)
    with pytest.raises(moon.MoonError):  # 48 is no multiple of 32
        moon.moon_mx4_quantize(torch.zeros((4, 48), device=dev), u8(4, 24), u8(4, 1))
    with pytest.raises(moon.MoonError):  # values not 16-byte aligned
        moon.moon_mx4_quantize(torch.zeros(257, device=dev)[1:].view(4, 64), u8(4, 32), u8(4, 2))
    arrays, NvS = ref.plan_arrays([[3, 2]], 1, 1)
    plan = {k: torch.from_numpy(v).to(dev) for k, v in arrays.items()}
    moon.moon_mx4_quantize(torch.zeros((NvS, 64), device=dev), u8(NvS, 32), u8(NvS, 2), plan=plan)
    plan["zero_fill_ranges"] = plan["zero_fill_ranges"][:, :1].contiguous()
    with pytest.raises(ValueError):
        moon.moon_mx4_quantize(x, u8(4, 32), u8(4, 2), plan=plan)


def test_rows_of_more_than_one_launch_could_cover(env):
    """2^30 + 5 rows of 32 values (64 + 16 GiB): with 64 rows a workgroup they
    would take more threads than a launch may have."""
    moon, torch, dev = env
    n = 2 ** 30 + 5
    say(f"[case] {n} rows")
    if torch.cuda.mem_get_info(dev)[0] < 90 * 2 ** 30:
        pytest.skip("needs 90 GiB")
    x = torch.full((n, 32), 1.5, dtype=torch.bfloat16, device=dev)
    x[-1] = -3.0
    q = torch.zeros((n, 16), dtype=torch.uint8, device=dev)
    s = torch.zeros((n, 1), dtype=torch.uint8, device=dev)
    moon.moon_mx4_quantize(x, q, s)
    del x
    torch.cuda.synchronize()
    words = q.view(torch.int64)  # 1.5 = 6 * 2^-2, -3 = -6 * 2^-1
    for a in range(0, n - 1, 2 ** 27):
        b = min(a + 2 ** 27, n - 1)
        assert bool((words[a:b] == 0x7777777777777777).all()) and bool((s[a:b] == 125).all())
    assert q[-1].tolist() == [0xFF] * 16 and s[-1].item() == 126
