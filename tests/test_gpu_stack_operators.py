"""The norm, the routing by scores and the dense products together, as a stack uses them: routed
layers with a routing rule (resident tables, with and without prefetch), dense layers with FP16 and
with 8-bit activations, the residual stream between them.  Every layer is checked on the input that
it had: norms and routing exactly, outputs against fp64 evaluations of the same weights."""
import numpy as np
import pytest

import oracle
from parity_util import f16_to_f64
from test_gpu_rmsnorm import EPS, expected as norm_expected
from test_gpu_route_scored import SIGMOID, TOP2, expected as route_expected
from w4a16_routed_expert_amd import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

RULE = dict(score=SIGMOID, n_group=4, topk_group=2, group=TOP2, scale=2.5)
DEV = "cuda:0"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def rule():
    from w4a16_routed_expert_amd import binding as B
    return B.route_rule(score=B.MOE_SCORE_SIGMOID, n_group=4, topk_group=2, group_score=B.MOE_GROUP_TOP2, scale=2.5)


def routed_output(cfg, rows, xn, want):
    """fp64 output of the routed experts `want` chose, h rounded to FP16 as the layer rounds it."""
    y = np.zeros((xn.shape[0], cfg.H))
    for e in np.unique(want["ids"]):
        Wg, Wu, Wd = oracle.dequant_expert(rows[e], cfg.H, cfg.I)
        t, j = np.nonzero(want["ids"] == e)
        x = xn[t].astype(np.float64)
        g, u = x @ Wg.T, x @ Wu.T
        h = (g / (1 + np.exp(-g)) * u).astype(np.float16).astype(np.float64)
        y[t] += want["w"][t, j].astype(np.float64)[:, None] * (h @ Wd.T)
    return y


def near(got, want, what):
    """FP16 outputs of two chained products: within 2^-8 of each row's largest value (h rounds to FP16,
    and values next to a rounding border round either way)."""
    d = np.abs(got.astype(np.float64) - want)
    tol = 2.0 ** -8 * np.abs(want).max(axis=1, keepdims=True) + 2.0 ** -20
    assert np.all(d <= tol), f"{what}: {(d / tol).max()} of the tolerance"


class Dense:
    def __init__(self, H, I, e4m3, seed):
        from w4a16_routed_expert_amd.layer import DenseFFN
        g = np.random.default_rng(seed)
        up = torch.from_numpy((g.standard_normal((I, H)) / np.sqrt(H)).astype(np.float32))
        self.scale = None
        if e4m3:
            self.scale = (up.abs().amax(1) / 448.0).float()
            up = (up / self.scale[:, None]).to(torch.float8_e4m3fn)
        else:
            up = up.half()
        self.up = up.double().numpy() * (1.0 if self.scale is None else self.scale.double().numpy()[:, None])
        down = (g.standard_normal((H, I)) / np.sqrt(I)).astype(np.float16)
        self.down, self.ub = down.astype(np.float64), (0.1 * g.standard_normal(I)).astype(np.float32)
        self.layer = DenseFFN(up.to(DEV), dev(down), None if self.scale is None else self.scale.to(DEV),
                              up_bias=dev(self.ub))

    def output(self, x, residual):
        z = x @ self.up.T + self.ub
        h = (z / (1 + np.exp(-z))).astype(np.float16).astype(np.float64)
        return h @ self.down.T + residual.astype(np.float64)


@pytest.mark.parametrize("T", [1, 3, 20, 70])
def test_norms_scored_layers_and_dense_layers_in_a_stack(T):
    from w4a16_routed_expert_amd.layer import DecodeStack, ResidentExpertTable, RoutedExpertLayer
    cfg = synth.CONFIGS["tiny"]
    H, E, k = cfg.H, cfg.E, cfg.k
    g = np.random.default_rng(T)
    kinds = ["routed", "dense", "routed", "dense8", "routed"]
    norms = [(1.0 + 0.2 * g.standard_normal(H)).astype(np.float16) for _ in kinds]
    outs = {}
    for prefetch in (False, True):
        layers, tables, host = [], [], []
        for l, kind in enumerate(kinds):
            if kind == "routed":
                rows, wr = synth.make_expert_rows(cfg, layer=l), synth.make_router(cfg, layer=l)
                bias = (0.1 * np.random.default_rng(l).standard_normal(E)).astype(np.float32)
                tab = ResidentExpertTable(rows, H, cfg.I, 4, 4, top_k=k, max_tokens=T)
                _, stride, _ = tab.device()
                layers.append(RoutedExpertLayer(H, cfg.I, E, k, torch.empty((1, stride), dtype=torch.uint8, device=DEV),
                                                dev(wr), max_T=T, rule=rule(), select_bias=dev(bias)))
                tables.append(tab)
                host.append((rows, wr, bias))
            else:
                d = Dense(H, 320, kind == "dense8", l)
                layers.append(d.layer)
                tables.append(None)
                host.append(d)
        stack = DecodeStack(layers, tables, prefetch=prefetch, norms=[dev(n) for n in norms], eps=EPS)
        steps = []
        for s in range(2):
            x0 = synth.make_x(cfg, T, step=40 + s)
            ys = []
            xL = stack.step(dev(x0), ys=ys)
            torch.cuda.synchronize()
            steps.append((x0, [y.cpu().numpy() for y in ys], xL.cpu().numpy()))
            last = {l: (layers[l].topk_ids[:T].cpu().numpy(), layers[l].topk_w[:T].cpu().numpy())
                    for l, kind in enumerate(kinds) if kind == "routed"}
        for l, kind in enumerate(kinds):
            if kind == "routed":
                layers[l].check_status()
                tables[l].close()
        outs[prefetch] = steps
    for (_, ya, xa), (_, yb, xb) in zip(outs[False], outs[True]):
        assert all(np.array_equal(a.view(np.uint16), b.view(np.uint16)) for a, b in zip(ya, yb))
        assert np.array_equal(xa.view(np.uint16), xb.view(np.uint16)), "prefetch changed the result"
    # the last step layer by layer, each on the input that it had
    x, ys, xL = outs[True][-1]
    for l, kind in enumerate(kinds):
        n = norm_expected(x, None, norms[l])
        if kind == "routed":
            rows, wr, bias = host[l]
            want = route_expected(oracle.router_logits(n["norm"], wr), k, bias, **RULE)
            ids, w = last[l]
            assert np.array_equal(ids, want["ids"]), f"layer {l}: experts"
            assert np.allclose(w, want["w"], rtol=2.0 ** -23, atol=0)
            near(ys[l], routed_output(cfg, rows, n["norm"], want), f"layer {l} (routed)")
            x = (f16_to_f64(x) + f16_to_f64(ys[l])).astype(np.float16)
        else:
            d = host[l]
            if kind == "dense8":
                q = torch.from_numpy(n["q"]).view(torch.float8_e4m3fn).double().numpy()
                xin = q * n["q_scale"].astype(np.float64)[:, None]
            else:
                xin = n["norm"].astype(np.float64)
            near(ys[l], d.output(xin, x), f"layer {l} ({kind})")
            x = ys[l]
    assert np.array_equal(x.view(np.uint16), xL.view(np.uint16)), "the residual stream"


def test_fused_and_shared_forwards_of_a_scored_layer():
    from w4a16_routed_expert_amd.layer import RoutedExpertLayer, SharedExpert
    cfg = synth.CONFIGS["tiny"]
    T = 6
    rows, wr, x = synth.make_expert_rows(cfg), synth.make_router(cfg), synth.make_x(cfg, T)
    g = np.random.default_rng(2)
    mats = [dev((g.standard_normal(s) * 0.05).astype(np.float16)) for s in ((128, cfg.H), (128, cfg.H), (cfg.H, 128),
                                                                           (cfg.H,))]
    lay = RoutedExpertLayer(cfg.H, cfg.I, cfg.E, cfg.k, dev(rows), dev(wr), max_T=T, rule=rule())
    want = route_expected(oracle.router_logits(x, wr), cfg.k, None, **RULE)
    a = lay.forward(dev(x))
    near(a.cpu().numpy(), routed_output(cfg, rows, x, want), "forward")
    assert torch.equal(a, lay.forward_fused(dev(x)))
    sh = SharedExpert(*mats, max_T=T)
    b = lay.forward(dev(x), shared=sh)
    assert torch.equal(b, lay.forward_fused(dev(x), shared=sh)) and torch.equal(b, lay.forward_shared(dev(x), sh))
    assert not torch.equal(a, b)
    with pytest.raises(ValueError):
        lay.route(dev(x), exact=True)
    with pytest.raises(ValueError):
        RoutedExpertLayer(cfg.H, cfg.I, cfg.E, cfg.k, dev(rows), dev(wr), bias=dev(np.zeros(cfg.E, np.float32)),
                          rule=rule())


def test_a_larger_batch_grows_the_buffers():
    from w4a16_routed_expert_amd.layer import RoutedExpertLayer
    cfg = synth.CONFIGS["tiny"]
    rows, wr = synth.make_expert_rows(cfg), synth.make_router(cfg)
    lay = RoutedExpertLayer(cfg.H, cfg.I, cfg.E, cfg.k, dev(rows), dev(wr), max_T=2, rule=rule())
    dense = Dense(cfg.H, 96, True, 9)
    for T in (2, 150, 30):
        x = synth.make_x(cfg, T, step=T)
        lay.route(dev(x))
        want = route_expected(oracle.router_logits(x, wr), cfg.k, None, **RULE)
        assert np.array_equal(lay.topk_ids[:T].cpu().numpy(), want["ids"])
        assert np.array_equal(lay.pair_pos[:T * cfg.k].cpu().numpy(), want["pair_pos"])
        n = norm_expected(x, None, np.ones(cfg.H, np.float16))
        q = torch.from_numpy(n["q"]).view(torch.float8_e4m3fn)
        got = dense.layer.run(q.to(DEV), dev(n["q_scale"]), residual=dev(x)).cpu().numpy()
        near(got, dense.output(q.double().numpy() * n["q_scale"].astype(np.float64)[:, None], x), f"T={T}")


class Block:
    """norm -> routed experts (scores) -> residual + norm to 8 bits -> dense layer, resident weights."""

    def __init__(self, cfg, T, seed=0):
        from w4a16_routed_expert_amd.layer import RoutedExpertLayer
        g = np.random.default_rng(seed)
        self.H, self.T = cfg.H, T
        self.w = [dev((1.0 + 0.2 * g.standard_normal(cfg.H)).astype(np.float16)) for _ in range(2)]
        self.lay = RoutedExpertLayer(cfg.H, cfg.I, cfg.E, cfg.k, dev(synth.make_expert_rows(cfg)),
                                     dev(synth.make_router(cfg)), max_T=T, rule=rule())
        self.dense = Dense(cfg.H, 320, True, seed).layer
        f16 = dict(dtype=torch.float16, device=DEV)
        self.n, self.y, self.s, self.out = (torch.empty((T, cfg.H), **f16) for _ in range(4))
        self.q = torch.empty((T, cfg.H), dtype=torch.float8_e4m3fn, device=DEV)
        self.scale = torch.empty(T, dtype=torch.float32, device=DEV)

    def run(self, x, stream=None):
        from w4a16_routed_expert_amd import binding as B
        T, H = self.T, self.H
        B.moe_residual_rmsnorm(x, None, self.w[0], EPS, T, H, norm=self.n, stream=stream)
        self.lay.forward(self.n, self.y, stream)
        B.moe_residual_rmsnorm(x, self.y, self.w[1], EPS, T, H, sum_out=self.s, q=self.q, q_scale=self.scale,
                               stream=stream)
        return self.dense.run(self.q, self.scale, residual=self.s, out=self.out, stream=stream)


@pytest.mark.parametrize("T", [1, 24, 90])
def test_a_block_captured_and_replayed(T):
    cfg = synth.CONFIGS["tiny"]
    b = Block(cfg, T)
    xs = [dev(synth.make_x(cfg, T, step=s)) for s in range(4)]
    want = [b.run(x).clone() for x in xs]
    x = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(x)
    for i in (2, 0, 3, 1, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.out, want[i]), f"replay on input {i}"
        assert torch.equal(b.run(xs[i]), want[i]), "an eager call between replays"
        torch.cuda.synchronize()


def test_blocks_on_streams_of_their_own():
    cfg = synth.CONFIGS["tiny"]
    T = 40
    blocks = [Block(cfg, T, seed=s) for s in range(2)]
    xs = [dev(synth.make_x(cfg, T, step=s)) for s in range(2)]
    want = [b.run(x).clone() for b, x in zip(blocks, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(8):
        for b, x, s in zip(blocks, xs, streams):
            b.out.zero_()
            s.wait_stream(torch.cuda.current_stream())
            b.run(x, s)
        torch.cuda.synchronize()
        for b, w in zip(blocks, want):
            assert torch.equal(b.out, w)


def test_buffers_that_grow_on_another_stream():
    from w4a16_routed_expert_amd.layer import RoutedExpertLayer
    cfg = synth.CONFIGS["tiny"]
    rows, wr = dev(synth.make_expert_rows(cfg)), dev(synth.make_router(cfg))
    lay = RoutedExpertLayer(cfg.H, cfg.I, cfg.E, cfg.k, rows, wr, max_T=1, rule=rule())
    dense = Dense(cfg.H, 160, False, 3).layer
    s = torch.cuda.Stream()
    for T in (1, 30, 100, 400):
        x = dev(synth.make_x(cfg, T, step=T))
        want = lay.__class__(cfg.H, cfg.I, cfg.E, cfg.k, rows, wr, max_T=T, rule=rule()).forward(x)
        ref = dense.run(x)
        s.wait_stream(torch.cuda.current_stream())
        y, d = lay.forward(x, stream=s), dense.run(x, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(d, ref)
