"""moe_residual_rmsnorm against its definition evaluated step by step on the host.

Every step after the fp64 sum is one IEEE FP32 operation, so the expected
values are exact: the stream, the FP16 norm, the scales and the 8-bit codes
are compared bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

EPS = 1e-5
BIG = 1 << 16                                        # elements that guard the ends of output buffers


def e4m3_bits(z):
    """Nearest e4m3 code of FP32 values |z| < 464 (ties to even), NaN -> 0x7f, by its definition."""
    z = np.asarray(z, np.float64)
    a = np.abs(np.where(np.isnan(z), 0.0, z))
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6.0)
    m = np.rint(a / 2.0 ** (e - 3))                  # 8..16 for normal values, 0..8 below 2^-6
    code = np.where(m >= 16, (e + 1 + 7) * 8, np.where(m >= 8, (e + 7) * 8 + (m - 8), m)).astype(np.int64)
    code = code + np.where(np.signbit(z), 128, 0)
    return np.where(np.isnan(z), 0x7F, code).astype(np.uint8)


def expected(x, y, w, eps=EPS):
    f = np.float32
    v = x if y is None else (x.astype(np.float64) + y.astype(np.float64)).astype(np.float16)
    v64 = v.astype(np.float64)
    ms = (v64 * v64).sum(axis=1) / x.shape[1]
    r = (1.0 / np.sqrt(ms + float(f(eps)))).astype(f)
    n = v.astype(f) * r[:, None] * w.astype(f)[None, :]
    assert n.dtype == f
    amax = np.abs(n).max(axis=1)                     # NaN if the row holds one
    a = np.where(np.isnan(amax), amax, np.maximum(amax, f(2.0 ** -100))).astype(f)
    q = e4m3_bits(n * (f(448.0) / a)[:, None])
    with np.errstate(over="ignore"):
        return dict(sum=v, norm=n.astype(np.float16), q_scale=a / f(448.0), q=q)


def same(got, want, what):
    for name, g in got.items():
        e = want[name]
        if g.dtype.kind == "f":
            nan = np.isnan(e)
            assert np.array_equal(np.isnan(g), nan), f"{what}: {name}: NaN places differ"
            bits = {2: np.uint16, 4: np.uint32}[g.itemsize]
            bad = (g.view(bits) != e.view(bits)) & ~nan
        else:
            bad = g != e
            if name == "q":                          # a NaN code keeps no sign
                bad &= ~(((g & 0x7F) == 0x7F) & ((e & 0x7F) == 0x7F))
        assert not bad.any(), f"{what}: {name} differs at {np.argwhere(bad)[:5].tolist()} of {g.shape}"


def run(x, y, w, want=("sum", "norm", "q"), eps=EPS, ld=None, offset=0, alias=None):
    """One call on copies; ld: row stride of every matrix; offset: elements before its first row;
    alias: the name of the output that is written over x."""
    from w4a16_routed_expert_amd import binding as B
    dev = torch.device("cuda:0")
    T, H = x.shape
    ld = H if ld is None else ld

    def place(a, dtype, fill=None):
        buf = torch.full((offset + max(T, 1) * ld + BIG,), 77, dtype=dtype, device=dev)
        view = buf[offset:offset + max(T, 1) * ld].view(max(T, 1), ld)[:T, :H]
        if a is not None:
            view.copy_(torch.from_numpy(np.ascontiguousarray(a)))
        return buf, view

    _, xv = place(x, torch.float16)
    yv = None if y is None else place(y, torch.float16)[1]
    wv = torch.from_numpy(w).to(dev)
    bufs = {n: place(None, torch.uint8 if n == "q" else torch.float16) for n in want}
    if alias:
        bufs[alias] = (None, xv)
    scale = torch.full((max(T, 1) + 8,), 77.0, dtype=torch.float32, device=dev) if "q" in want else None
    B.moe_residual_rmsnorm(xv, yv, wv, eps, T, H, sum_out=bufs["sum"][1] if "sum" in want else None,
                           norm=bufs["norm"][1] if "norm" in want else None,
                           q=bufs["q"][1] if "q" in want else None, q_scale=scale, ldx=ld, ldy=ld, ld_sum=ld,
                           ld_norm=ld, ldq=ld)
    torch.cuda.synchronize()
    got = {}
    for n, (buf, view) in bufs.items():
        got[n] = view.cpu().numpy()
        if buf is not None:                          # nothing outside the rows is written
            rest = torch.ones_like(buf, dtype=torch.bool)
            rest[offset:offset + max(T, 1) * ld].view(max(T, 1), ld)[:T, :H] = False
            assert bool((buf[rest] == 77).all()), f"{n}: written outside its rows"
    if scale is not None:
        assert bool((scale[T:] == 77.0).all())
        got["q_scale"] = scale[:T].cpu().numpy()
    return got


def inputs(T, H, seed=0):
    g = np.random.default_rng([seed, T, H])
    x = (g.standard_normal((T, H)) * np.exp(g.standard_normal(H))).astype(np.float16)
    y = g.standard_normal((T, H)).astype(np.float16)
    w = (1.0 + 0.2 * g.standard_normal(H)).astype(np.float16)
    return x, y, w


@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (5, 8), (4, 9), (2, 511), (7, 512), (3, 513), (5, 1024), (2, 1411),
                                 (1, 2048), (33, 2048), (3, 2049), (5, 4096), (2, 4100), (3, 8192), (2, 8200),
                                 (2, 16384), (1, 16391), (1, 65536)])
def test_equals_the_definition(T, H):
    x, y, w = inputs(T, H)
    want = expected(x, y, w)
    same(run(x, y, w), want, f"T={T} H={H}")
    alone = expected(x, None, w)
    for names in (("norm",), ("q",), ("sum",), ("norm", "q")):
        same(run(x, None, w, names), alone, f"T={T} H={H} {names}, no addition")


@pytest.mark.parametrize("H,ld,offset", [(256, 264, 0), (256, 257, 1), (1411, 1500, 3), (2048, 4096, 8), (2050, 2051, 5)])
def test_strided_and_unaligned_rows(H, ld, offset):
    x, y, w = inputs(6, H, 1)
    same(run(x, y, w, ld=ld, offset=offset), expected(x, y, w), f"H={H} ld={ld} offset={offset}")


@pytest.mark.parametrize("H", [13, 512, 2048, 4100])
@pytest.mark.parametrize("alias", ["sum", "norm"])
def test_outputs_may_replace_x(H, alias):
    x, y, w = inputs(9, H, 2)
    same(run(x, y, w, alias=alias), expected(x, y, w), f"H={H} {alias} over x")


@pytest.mark.parametrize("H", [8, 640, 2048, 4096])
def test_special_rows(H):
    x, y, w = inputs(8, H, 3)
    x[0], y[0] = 0, 0                                # nothing in the row: codes 0, a small scale
    x[1, :] = 6e-8                                   # smallest subnormals
    y[1, :] = 0
    x[2, 3] = np.inf
    x[3, H - 1] = np.nan
    x[4, 0], y[4, 0] = 65504, 65504                  # the addition overflows
    x[5, :], y[5, :] = 65504, 0                      # the sum of squares passes FP16 and FP32 sums of FP16 squares
    x[6, :], y[6, :] = 1.0, -1.0 + 2.0 ** -11        # cancellation
    w[H // 2] = 0
    with np.errstate(invalid="ignore", over="ignore"):
        want = expected(x, y, w)
        got = run(x, y, w)
    same(got, want, f"H={H}")
    assert not got["q"][0].any() and got["q_scale"][0] > 0


def test_zero_rows_of_tokens_enqueue_nothing():
    x, y, w = inputs(0, 64)
    assert run(x, y, w)["norm"].shape == (0, 64)


def test_no_tie_to_the_largest_code():
    # n * RN32(448 / a) may pass 448 by one FP32 step: still the code of 448
    H = 64
    g = np.random.default_rng(5)
    x = (g.standard_normal((4096, H)) * np.exp(g.uniform(-4, 4, (4096, 1)))).astype(np.float16)
    w = np.ones(H, np.float16)
    got = run(x, None, w, ("q",))
    same(got, expected(x, None, w), "codes")
    assert np.all((got["q"] & 0x7F).max(axis=1) == 0x7E)


def test_offsets_past_32_bits():
    # 70,000 rows 40,000 elements apart: 5.6 GB, rows past 2^31 elements
    from w4a16_routed_expert_amd import binding as B
    dev = torch.device("cuda:0")
    T, H, ld = 70000, 24, 40000
    x, _, w = inputs(T, H, 6)
    buf = torch.zeros(T * ld, dtype=torch.float16, device=dev)
    view = buf.view(T, ld)[:, :H]
    view.copy_(torch.from_numpy(x))
    norm = torch.empty((T, H), dtype=torch.float16, device=dev)
    B.moe_residual_rmsnorm(view, None, torch.from_numpy(w).to(dev), EPS, T, H, norm=norm)
    torch.cuda.synchronize()
    same({"norm": norm.cpu().numpy()}, expected(x, None, w), "far rows")


def test_captured_and_on_another_stream():
    from w4a16_routed_expert_amd import binding as B
    dev = torch.device("cuda:0")
    T, H = 17, 2048
    x, y, w = inputs(T, H, 7)
    xd, yd, wd = (torch.from_numpy(a).to(dev) for a in (x, y, w))
    out = {"sum": torch.empty_like(xd), "norm": torch.empty_like(xd)}
    q, scale = torch.empty((T, H), dtype=torch.uint8, device=dev), torch.empty(T, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.moe_residual_rmsnorm(xd, yd, wd, EPS, T, H, sum_out=out["sum"], norm=out["norm"], q=q, q_scale=scale)
    for step in range(3):
        x2, y2, _ = inputs(T, H, 8 + step)
        xd.copy_(torch.from_numpy(x2))
        yd.copy_(torch.from_numpy(y2))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.cpu().numpy() for n, t in (*out.items(), ("q", q), ("q_scale", scale))}
        same(got, expected(x2, y2, w), f"replay {step}")


@pytest.mark.parametrize("T,H", [(256, 1024), (257, 1024), (300, 513), (1001, 777), (260, 1000), (5000, 512), (3000, 2048)])
def test_longer_batches(T, H):
    test_equals_the_definition(T, H)
