"""CPU checks of the operators around the routed experts: their host-side validation rejects
bad arguments before touching a GPU, and empty batches are accepted."""
import pytest

from w4a16_routed_expert_amd import binding as B

F = 0x1000  # never dereferenced: validation fails first


def refused(call, code, word):
    with pytest.raises(B.MoeError) as ei:
        call()
    assert ei.value.code == code, B.moe_last_error()
    assert word in B.moe_last_error(), B.moe_last_error()


def norm(x=F, y=F, w=F, eps=1e-5, T=4, H=256, **kw):
    out = dict(sum_out=F * 2, norm=F * 3, q=F * 4, q_scale=F * 5)
    out.update(kw)
    B.moe_residual_rmsnorm(x, y, w, eps, T, H, stream=0, **out)


def test_rmsnorm_refusals():
    for kw in (dict(T=-1), dict(H=0), dict(H=65537), dict(H=-8)):
        refused(lambda: norm(**kw), B.MOE_ERR_UNSUPPORTED, "H=")
    for eps in (0.0, -1e-5, 2.0, float("nan"), float("inf")):
        refused(lambda: norm(eps=eps), B.MOE_ERR_INVALID_ARG, "eps")
    refused(lambda: norm(x=None), B.MOE_ERR_INVALID_ARG, "null")
    refused(lambda: norm(w=None), B.MOE_ERR_INVALID_ARG, "null")
    refused(lambda: norm(sum_out=None, norm=None, q=None, q_scale=None), B.MOE_ERR_INVALID_ARG, "no output")
    refused(lambda: norm(q=None), B.MOE_ERR_INVALID_ARG, "q_scale")
    refused(lambda: norm(q_scale=None), B.MOE_ERR_INVALID_ARG, "q_scale")
    for ld in ("ldx", "ldy", "ld_sum", "ld_norm", "ldq"):
        refused(lambda: norm(**{ld: 255}), B.MOE_ERR_INVALID_ARG, "stride")
    for kw in (dict(x=F + 1), dict(y=F + 1), dict(w=F + 1), dict(sum_out=F + 1), dict(norm=F + 1),
               dict(q_scale=F + 2)):
        refused(lambda: norm(**kw), B.MOE_ERR_INVALID_ARG, "aligned")
    refused(lambda: norm(norm=F * 2), B.MOE_ERR_INVALID_ARG, "same buffer")
    norm(T=0, x=None, y=None, w=None)                # nothing to do


def scored(T=4, H=256, E=8, k=2, x=F, wr=F, ids=F, ws=F, ws_bytes=1 << 20, rule="default", bias=None, **r):
    if rule == "default":
        rule = B.route_rule(**r)
    B.moe_route_scored(x, wr, bias, T, H, E, k, rule, None, ids, F, F, F, F, F, F, ws, ws_bytes, stream=0)


def test_scored_routing_refusals():
    for kw in (dict(E=65), dict(E=0, k=1), dict(k=9), dict(k=0), dict(T=-1), dict(T=65537), dict(H=200), dict(H=0),
               dict(H=4224)):
        refused(lambda: scored(**kw), B.MOE_ERR_UNSUPPORTED, "=")
    refused(lambda: scored(rule=None), B.MOE_ERR_INVALID_ARG, "rule")
    refused(lambda: scored(bias=F + 2), B.MOE_ERR_INVALID_ARG, "aligned")
    refused(lambda: scored(x=F + 8), B.MOE_ERR_INVALID_ARG, "aligned")
    for kw, word in ((dict(score=2), "score"), (dict(score=-1), "score"), (dict(group_score=2), "group score"),
                     (dict(n_group=3), "n_group"), (dict(n_group=0), "n_group"), (dict(n_group=16), "n_group"),
                     (dict(n_group=4, topk_group=5), "topk_group"), (dict(n_group=4, topk_group=0), "topk_group"),
                     (dict(n_group=8, topk_group=1), "exceeds"), (dict(scale=0.0), "scale"),
                     (dict(scale=-1.0), "scale"), (dict(scale=float("nan")), "scale"),
                     (dict(scale=float("inf")), "scale"),
                     (dict(n_group=8, topk_group=2, group_score=B.MOE_GROUP_TOP2), "two largest")):
        refused(lambda: scored(**kw), B.MOE_ERR_INVALID_ARG, word)
    for kw in (dict(x=None), dict(wr=None), dict(ids=None)):
        refused(lambda: scored(**kw), B.MOE_ERR_INVALID_ARG, "null")
    refused(lambda: scored(x=F + 8), B.MOE_ERR_INVALID_ARG, "aligned")
    refused(lambda: scored(wr=F + 1), B.MOE_ERR_INVALID_ARG, "aligned")
    need = B.moe_route_scored_workspace_size(4, 256, 8)
    for kw in (dict(ws=None), dict(ws_bytes=need - 1), dict(ws=F + 128)):
        refused(lambda: scored(**kw), B.MOE_ERR_WORKSPACE, "workspace")
    scored(T=0, x=None)                              # nothing to do


def test_scored_routing_workspace_serves_smaller_batches():
    for E in (1, 8, 60, 64):
        sizes = [B.moe_route_scored_workspace_size(T, 2048, E) for T in [*range(0, 300), 1000, 4096, 65536]]
        assert all(b >= a for a, b in zip(sizes, sizes[1:])) and all(s % 256 == 0 and s >= 256 for s in sizes)
    assert B.moe_route_scored_workspace_size(4, 2048, 65) == 0
    assert B.moe_route_scored_workspace_size(65537, 2048, 8) == 0


def test_row_strides_of_tensors():
    import torch
    base = torch.zeros(10, 32, dtype=torch.float16)
    assert B._ld(base, None, 32) == 32 and B._ld(base[:, :24], None, 24) == 32 and B._ld(base[::2], None, 32) == 64
    assert B._ld(base[:1], None, 32) == 32 and B._ld(base[0], None, 32) == 32 and B._ld(F, None, 8) == 8
    assert B._ld(base, 77, 32) == 77 and B._ld(None, None, 5) == 5
    with pytest.raises(ValueError):
        B._ld(base.t(), None, 10)


def linear(T=4, N=64, K=128, type=B.MOE_LINEAR_FP16, x=F, w=F, y=F, ws=F, ws_bytes=1 << 30, **kw):
    B.moe_linear(x, w, T, N, K, type, y, ws=ws, ws_bytes=ws_bytes, stream=0, **kw)


def test_linear_refusals():
    E4M3 = B.MOE_LINEAR_E4M3
    refused(lambda: linear(type=2), B.MOE_ERR_INVALID_ARG, "type")
    refused(lambda: linear(act=4), B.MOE_ERR_INVALID_ARG, "activation")
    refused(lambda: linear(act=-1), B.MOE_ERR_INVALID_ARG, "activation")
    for kw in (dict(T=-1), dict(T=65537), dict(N=0), dict(N=(1 << 24) + 1), dict(K=0), dict(K=8), dict(K=24),
               dict(K=(1 << 20) + 16)):
        refused(lambda: linear(**kw), B.MOE_ERR_UNSUPPORTED, "=")
    for kw in (dict(x=None), dict(w=None), dict(y=None)):
        refused(lambda: linear(**kw), B.MOE_ERR_INVALID_ARG, "null")
    for kw in (dict(x_scale=F), dict(w_scale=F), dict(x_scale=F, w_scale=F), dict(type=E4M3),
               dict(type=E4M3, x_scale=F), dict(type=E4M3, w_scale=F)):
        refused(lambda: linear(**kw), B.MOE_ERR_INVALID_ARG, "scale")
    for kw in (dict(ldx=112), dict(ldw=112), dict(ldy=63), dict(residual=F, ldr=63)):
        refused(lambda: linear(**kw), B.MOE_ERR_INVALID_ARG, "stride")
    for kw in (dict(ldx=(1 << 22) + 16), dict(ldw=(1 << 22) + 16)):
        refused(lambda: linear(**kw), B.MOE_ERR_UNSUPPORTED, "strides")
    for kw in (dict(x=F + 8), dict(w=F + 8), dict(ldx=132), dict(ldw=132)):
        refused(lambda: linear(**kw), B.MOE_ERR_INVALID_ARG, "16 bytes")
    refused(lambda: linear(type=E4M3, x_scale=F, w_scale=F, ldx=136), B.MOE_ERR_INVALID_ARG, "16 bytes")
    for kw in (dict(y=F + 1), dict(residual=F + 1), dict(bias=F + 2)):
        refused(lambda: linear(**kw), B.MOE_ERR_INVALID_ARG, "aligned")
    need = B.moe_linear_workspace_size(4, 64, 128, B.MOE_LINEAR_FP16)
    for kw in (dict(ws=None), dict(ws_bytes=need - 1), dict(ws=F + 16)):
        refused(lambda: linear(**kw), B.MOE_ERR_WORKSPACE, "workspace")
    for args in ((-1, 8, 16, 0), (4, 0, 16, 0), (4, 8, 8, 0), (4, 8, 24, 1), (4, 8, 16, 2)):
        assert B.moe_linear_workspace_size(*args) == 0
    linear(T=0, x=None, w=None, y=None, ws=None, ws_bytes=0)    # nothing to do


def test_host_tensors_are_refused():
    # a host address would fault the GPU: refused before anything is enqueued
    import torch
    h = torch.zeros(4, 256, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU memory"):
        B.moe_residual_rmsnorm(h, None, F, 1e-5, 4, 256, norm=F, stream=0)
    with pytest.raises(ValueError, match="one GPU"):
        B.moe_residual_rmsnorm(F, None, h, 1e-5, 4, 256, norm=F, stream=0)
    with pytest.raises(ValueError, match="GPU memory"):
        B.moe_linear(h, F, 4, 64, 256, B.MOE_LINEAR_FP16, F, ws=F, ws_bytes=1 << 30, stream=0)
    with pytest.raises(ValueError, match="one GPU"):
        B.moe_route_scored(F, h, None, 4, 256, 8, 2, B.route_rule(), None, F, F, F, F, F, F, F, F, 1 << 20, stream=0)


def test_layers_refuse_weights_of_other_shapes():
    torch = pytest.importorskip("torch")
    from w4a16_routed_expert_amd.layer import DecodeStack, DenseFFN, RoutedExpertLayer
    up, down = torch.zeros(96, 64, dtype=torch.float16), torch.zeros(64, 96, dtype=torch.float16)
    f8 = up.to(torch.float8_e4m3fn)
    f32 = torch.zeros(96)
    for args, kw in (((up.float(), down), {}), ((up, down.float()), {}), ((up, down.t()[:, :32]), {}),
                     ((up, down), dict(up_scale=f32)), ((f8, down), {}), ((f8, down), dict(up_scale=f32[:95])),
                     ((f8, down), dict(up_scale=f32.half())),
                     ((up, down), dict(up_bias=f32[:64])), ((up, down), dict(down_bias=f32)),
                     ((up, down), dict(up_bias=torch.zeros(192)[::2]))):
        with pytest.raises(ValueError):
            DenseFFN(*args, **kw)
    rule = B.route_rule(score=B.MOE_SCORE_SIGMOID)
    for kw in (dict(rule=rule, bias=f32), dict(select_bias=f32), dict(rule=rule, select_bias=f32[:7]),
               dict(rule=rule, select_bias=torch.zeros(8).double())):
        with pytest.raises(ValueError):
            RoutedExpertLayer(256, 256, 8, 2, torch.zeros(1, 1, dtype=torch.uint8), up, **kw)

    class Layer:
        H, device = 64, "cpu"
    for norms in ([f32[:64].half()], [f32[:64].half(), f32.half()], [f32[:64].half(), f32[:64]]):
        with pytest.raises(ValueError):
            DecodeStack([Layer(), Layer()], [None, None], norms=norms)
