"""moe_linear against its definition.

Whole-number inputs small enough that every partial sum is exact in FP32: the
result is then one rounding of an exact value, whatever the order of the sum,
and is compared bit for bit.  Random inputs: with P = sum |s x w| + |bias|, an
FP32 sum of K products in any order, each addition off by at most a step
(2^-23), is within (K + 2) 2^-23 P of the exact one; the activations' slope is
at most 1.13 and their FP32 evaluation (exp, erf, a division, a few products)
within 2^-19 of the value's size; the output rounds by half an FP16 step
(2^-11 relative, 2^-25 below the normal range)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NONE, SILU, GELU, GELU_TANH = 0, 1, 2, 3
FP16, E4M3 = 0, 1
GUARD = 1 << 14


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")


class Case:
    def __init__(self, T, N, K, type, whole, bias=True, res=True, seed=0):
        g = np.random.default_rng([seed, T, N, K, type])
        self.T, self.N, self.K, self.type = T, N, K, type
        if whole:
            self.x = g.integers(-4, 5, (T, K)).astype(np.float32)
            self.w = g.integers(-4, 5, (N, K)).astype(np.float32)
            self.bias = g.integers(-9, 10, N).astype(np.float32) if bias else None
            self.res = g.integers(-9, 10, (T, N)).astype(np.float16) if res else None
            self.sx = 2.0 ** g.integers(-1, 2, T).astype(np.float32) if type == E4M3 else None
            self.sw = 2.0 ** g.integers(-1, 2, N).astype(np.float32) if type == E4M3 else None
        else:
            self.x = g.standard_normal((T, K)).astype(np.float32)
            self.w = (g.standard_normal((N, K)) / math.sqrt(K)).astype(np.float32)
            self.bias = g.standard_normal(N).astype(np.float32) if bias else None
            self.res = g.standard_normal((T, N)).astype(np.float16) if res else None
            self.sx = g.uniform(0.5, 2, T).astype(np.float32) if type == E4M3 else None
            self.sw = g.uniform(0.5, 2, N).astype(np.float32) if type == E4M3 else None
            if type == E4M3:
                self.w *= np.float32(8.0)             # away from the subnormal codes
        t = torch.float16 if type == FP16 else torch.float8_e4m3fn
        self.xd = torch.from_numpy(self.x).to(t)
        self.wd = torch.from_numpy(self.w).to(t)
        self.x, self.w = self.xd.double().numpy(), self.wd.double().numpy()

    def run(self, act=NONE, ldx=None, ldw=None, ldy=None, offset=0, in_place=False, stream=None):
        from w4a16_routed_expert_amd import binding as B
        T, N, K = self.T, self.N, self.K
        ldx, ldw, ldy = ldx or K, ldw or K, ldy or N

        def rows(a, n, ld, width, fill, off=0):
            buf = torch.full((off + n * ld + GUARD,), fill, dtype=torch.float32, device="cuda:0").to(a.dtype)
            view = buf[off:off + n * ld].view(n, ld)[:, :width]
            view.copy_(a)
            return buf, view

        _, x = rows(self.xd, T, ldx, K, float("nan"))   # what lies between and behind rows must not matter
        _, w = rows(self.wd, N, ldw, K, float("nan"))
        res = None if self.res is None else rows(torch.from_numpy(self.res), T, ldy, N, 3.0, offset)[1]
        buf, y = rows(torch.zeros(T, N, dtype=torch.float16), T, ldy, N, 77.0, offset)
        if in_place:
            y.copy_(res)
            res = y
        need = B.moe_linear_workspace_size(T, N, K, self.type)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda:0")
        B.moe_linear(x, w, T, N, K, self.type, y, x_scale=dev(self.sx), w_scale=dev(self.sw), bias=dev(self.bias),
                     act=act, residual=res, ws=ws, ws_bytes=need, ldx=ldx, ldw=ldw, ldr=ldy, ldy=ldy, stream=stream)
        torch.cuda.synchronize()
        rest = torch.ones_like(buf, dtype=torch.bool)
        rest[offset:offset + T * ldy].view(T, ldy)[:, :N] = False
        assert bool((buf[rest] == 77.0).all()), "written outside the rows"
        return y.cpu().numpy()

    def expected(self, act=NONE):
        """(value in 64 bits, the tolerance of the module's text)."""
        s = 1.0 if self.sx is None else self.sx.astype(np.float64)[:, None] * self.sw.astype(np.float64)[None, :]
        z = (self.x @ self.w.T) * s
        p = (np.abs(self.x) @ np.abs(self.w).T) * s
        if self.bias is not None:
            z = z + self.bias.astype(np.float64)
            p = p + np.abs(self.bias)
        if act == SILU:
            v = z / (1 + np.exp(-z))
        elif act in (GELU, GELU_TANH):
            if act == GELU:
                v = torch.special.ndtr(torch.from_numpy(z)).numpy() * z
            else:
                v = 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        else:
            v = z
        tol = 1.13 * (self.K + 2) * 2.0 ** -23 * p + (2.0 ** -19 * np.abs(z) if act else 0.0)
        if self.res is not None:
            v = v + self.res.astype(np.float64)
            tol = tol + 2.0 ** -23 * np.abs(v)
        return v, tol + 2.0 ** -11 * (np.abs(v) + tol) + 2.0 ** -25

    def check_whole(self, got, what):
        want = self.expected()[0].astype(np.float16)
        bad = got.view(np.uint16) != want.view(np.uint16)
        bad &= ~((got == 0) & (want == 0))
        assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} differ, first {np.argwhere(bad)[:4].tolist()}"

    def check(self, got, act, what):
        v, tol = self.expected(act)
        off = np.abs(got.astype(np.float64) - v)
        bad = ~(off <= tol)
        assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(off / tol)} of the tolerance"


SHAPES = [(1, 1, 16), (1, 2048, 2048), (2, 17, 32), (3, 100, 48), (15, 16, 64), (16, 63, 128), (17, 65, 144),
          (31, 250, 1040), (32, 64, 4096), (33, 129, 2064), (48, 1411, 80), (63, 30, 112), (64, 257, 512),
          (65, 64, 16), (65, 1, 2048), (100, 333, 272), (127, 129, 1424), (129, 70, 64), (200, 640, 96), (256, 256, 8192),
          (333, 1411, 176), (700, 515, 208), (1900, 1921, 80), (2049, 1700, 64), (4000, 3700, 144), (2700, 2000, 96),
          (33, 70, 16384), (130, 90, 16400), (17, 300, 24576)]


@pytest.mark.parametrize("type", [FP16, E4M3], ids=["fp16", "e4m3"])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_whole_numbers_are_exact(T, N, K, type):
    c = Case(T, N, K, type, whole=True)
    c.check_whole(c.run(), f"{T}x{N}x{K}")
    c.bias = None
    c.check_whole(c.run(ldy=N + 1 + N % 2), f"{T}x{N}x{K} odd stride")
    c.res = None
    c.check_whole(c.run(), f"{T}x{N}x{K} plain")


@pytest.mark.parametrize("type", [FP16, E4M3], ids=["fp16", "e4m3"])
@pytest.mark.parametrize("act", [NONE, SILU, GELU, GELU_TANH], ids=["none", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T,N,K", [(1, 512, 2048), (9, 96, 1040), (40, 130, 512), (150, 257, 1424), (1000, 1300, 272)])
def test_random_values_and_activations(T, N, K, act, type):
    for bias, res in ((True, False), (False, True)):
        c = Case(T, N, K, type, whole=False, bias=bias, res=res)
        c.check(c.run(act), act, f"{T}x{N}x{K} act {act}")


@pytest.mark.parametrize("type", [FP16, E4M3], ids=["fp16", "e4m3"])
@pytest.mark.parametrize("T,N,K", [(1, 64, 128), (20, 100, 208), (70, 130, 80), (300, 1500, 64), (2000, 1999, 48)])
def test_strides_offsets_and_in_place(T, N, K, type):
    c = Case(T, N, K, type, whole=True)
    c.check_whole(c.run(ldx=K + 16, ldw=2 * K, ldy=N + 3, offset=1), "strided, unaligned")
    c.check_whole(c.run(ldx=K + 48, ldw=K + 16, ldy=(N + 7) // 4 * 4, offset=4), "strided, aligned")
    c.check_whole(c.run(in_place=True), "y over the residual")


@pytest.mark.parametrize("type", [FP16, E4M3], ids=["fp16", "e4m3"])
@pytest.mark.parametrize("T", [5, 50, 140, 2100])
def test_infinities_and_nans_stay_in_their_row(T, type):
    N, K = 1900 if T > 2000 else 200, 144
    c = Case(T, N, K, type, whole=True, bias=False, res=False)
    want = c.expected()[0].astype(np.float16)
    c.xd[T - 2, K - 1] = float("nan")
    c.wd[N - 3, 0] = float("nan")
    if type == FP16:
        c.xd[1, 5] = float("inf")
    got = c.run()
    assert np.isnan(got[T - 2]).all() and np.isnan(got[:, N - 3]).all()
    rows = [t for t in range(T) if t not in (T - 2, 1)]
    cols = [n for n in range(N) if n != N - 3]
    assert np.array_equal(got[np.ix_(rows, cols)] + 0.0, want[np.ix_(rows, cols)] + 0.0)
    if type == FP16:
        assert not np.isfinite(got[1]).any()


def test_activation_limits():
    # far values: no NaN where exp overflows; the limits are 0 and the value itself
    from w4a16_routed_expert_amd import binding as B
    K = 16
    z = np.array([-60000.0, -200.0, -90.0, -20.0, -0.0, 0.0, 20.0, 90.0, 60000.0], np.float16)
    x = np.zeros((z.size, K), np.float16)
    x[:, 0] = z
    w = np.zeros((1, K), np.float16)
    w[0, 0] = 1
    ws = torch.empty(B.moe_linear_workspace_size(z.size, 1, K, FP16), dtype=torch.uint8, device="cuda:0")
    for act in (SILU, GELU, GELU_TANH):
        y = torch.empty((z.size, 1), dtype=torch.float16, device="cuda:0")
        B.moe_linear(dev(x), dev(w), z.size, 1, K, FP16, y, act=act, ws=ws, ws_bytes=ws.numel())
        got = y.cpu().numpy()[:, 0].astype(np.float64)
        v = z.astype(np.float64)
        lo, hi = got[v < -50], got[v > 10]
        assert np.array_equal(lo, np.zeros_like(lo)) and np.array_equal(hi, v[v > 10])
        assert np.all(np.abs(got[(v >= -50) & (v <= 0)]) <= 1e-6)


def test_empty_batch_and_rows_past_2_gib():
    from w4a16_routed_expert_amd import binding as B
    B.moe_linear(None, None, 0, 8, 16, FP16, None)
    # x rows 2^20 elements apart: the last rows start past 2^31 bytes
    T, N, K, ld = 1500, 130, 64, 1 << 20
    g = np.random.default_rng(3)
    x = g.integers(-4, 5, (T, K)).astype(np.float16)
    w = g.integers(-4, 5, (N, K)).astype(np.float16)
    buf = torch.empty(T * ld, dtype=torch.float16, device="cuda:0")
    view = buf.view(T, ld)[:, :K]
    view.copy_(torch.from_numpy(x))
    y = torch.empty((T, N), dtype=torch.float16, device="cuda:0")
    ws = torch.empty(B.moe_linear_workspace_size(T, N, K, FP16), dtype=torch.uint8, device="cuda:0")
    B.moe_linear(view, dev(w), T, N, K, FP16, y, ws=ws, ws_bytes=ws.numel())
    assert np.array_equal(y.cpu().numpy().astype(np.float64), x.astype(np.float64) @ w.astype(np.float64).T)


@pytest.mark.parametrize("T,N,K", [(4, 640, 1024), (90, 200, 2048), (300, 300, 512), (40, 130, 8192), (1100, 900, 512)])
def test_captured_replays_and_repeated_calls(T, N, K):
    from w4a16_routed_expert_amd import binding as B
    c = Case(T, N, K, FP16, whole=False)
    x, w, b, r = (dev(a) for a in (c.xd.numpy(), c.wd.numpy(), c.bias, c.res))
    y = torch.empty((T, N), dtype=torch.float16, device="cuda:0")
    ws = torch.full((B.moe_linear_workspace_size(T, N, K, FP16),), 0xFF, dtype=torch.uint8, device="cuda:0")

    def call(out):
        B.moe_linear(x, w, T, N, K, FP16, out, bias=b, residual=r, act=SILU, ws=ws, ws_bytes=ws.numel())

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(y)
    for step in range(3):
        x.copy_(dev(Case(T, N, K, FP16, whole=False, seed=step + 1).xd.numpy()))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.empty_like(y)
        call(eager)
        torch.cuda.synchronize()
        assert torch.equal(y, eager), "a replay differs from the eager call"
        c.x = x.double().cpu().numpy()
        c.check(eager.cpu().numpy(), SILU, f"replay {step}")


@pytest.mark.parametrize("type", [FP16, E4M3], ids=["fp16", "e4m3"])
@pytest.mark.parametrize("T,N,K", [(1, 4111, 256), (5, 4100, 1040), (16, 5000, 2064), (9, 8193, 1040), (8, 8200, 1104),
                                   (13, 9001, 2064), (16, 4097, 4112)])
def test_few_tokens_and_many_outputs(T, N, K, type):
    c = Case(T, N, K, type, whole=True)
    c.check_whole(c.run(), f"{T}x{N}x{K}")
    c.check_whole(c.run(ldx=K + 16, ldw=K + 48, ldy=N + 3, offset=1), f"{T}x{N}x{K} strided")


@pytest.mark.parametrize("type", [FP16, E4M3], ids=["fp16", "e4m3"])
def test_many_tokens_and_outputs_with_a_long_sum(type):
    c = Case(3990, 3993, 4112, type, whole=True)
    c.check_whole(c.run(), "3990x3993x4112")
    c = Case(3990, 3985, 4112, type, whole=False)
    c.check(c.run(SILU), SILU, "3990x3985x4112 silu")


@pytest.mark.parametrize("type", [FP16, E4M3], ids=["fp16", "e4m3"])
@pytest.mark.parametrize("T,N,K", [(1, 17, 1 << 20), (16, 33, 1 << 20), (40, 70, 1 << 20), (65536, 5, 16), (65536, 67, 48),
                                   (1, 1 << 20, 16), (18, 1 << 18, 32)])
def test_the_largest_sizes(T, N, K, type):
    c = Case(T, N, K, type, whole=True)
    c.check_whole(c.run(), f"{T}x{N}x{K}")
