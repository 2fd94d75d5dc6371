"""Measured cases of the operators around the routed experts: the residual addition with its
root-mean-square norm (FP16 and 8-bit outputs), the routing by scores, and the dense matrix product
with its epilogue.

run() computes a case in elementary torch operations, or, with `own` set, through the library's
entry points (moe_residual_rmsnorm, moe_route_scored, moe_linear) on buffers that the state keeps.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
EPS = 1e-5
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100

# What the cases stand for in use:
#   norm_*    the step between two layers: the stack's residual addition and the next layer's norm.
#     norm_token       one token decoding, FP16 output
#     norm_ragged      a batch of requests at a hidden size that no vector width divides, norm only
#     norm_batch_e4m3  a decode batch whose dense layer takes 8-bit activations (codes and scales only)
#     norm_prompt      a long prompt: new residual stream, FP16 norm (router) and 8-bit norm (dense)
#   route_*   the router of a layer and the grouping its experts read.
#     route_token      one token, softmax over all 64 experts, weights renormalised
#     route_batch      a decode batch, sigmoid scores with a balance bias, 4 of 8 groups
#     route_ragged     60 experts in 4 groups by their best expert, a few hundred tokens
#     route_prompt     a long prompt, sigmoid scores, bias, groups
#   linear_*  the dense layers of a stack.
#     linear_token     one token through an FP16 projection added to the residual stream
#     linear_batch     a decode batch through an 8-bit up projection with SiLU
#     linear_ragged    a ragged prompt, odd output width, GELU, bias and residual
#     linear_prompt    a long prompt through 8-bit weights


def listed():
    return [
        dict(name="norm_token", op="norm", T=1, H=2048, add=True, fp16=True, e4m3=False),
        dict(name="norm_ragged", op="norm", T=333, H=1411, add=False, fp16=True, e4m3=False),
        dict(name="norm_batch_e4m3", op="norm", T=32, H=2048, add=True, fp16=False, e4m3=True),
        dict(name="norm_prompt", op="norm", T=8192, H=4096, add=True, fp16=True, e4m3=True),
        dict(name="route_token", op="route", T=1, H=2048, E=64, k=8, score="softmax", bias=False, n_group=1,
             topk_group=1, group="max", renorm=True, scale=1.0),
        dict(name="route_batch", op="route", T=32, H=2048, E=64, k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group="top2", renorm=True, scale=2.5),
        dict(name="route_ragged", op="route", T=611, H=1408, E=60, k=4, score="softmax", bias=False, n_group=4,
             topk_group=2, group="max", renorm=False, scale=1.0),
        dict(name="route_prompt", op="route", T=4096, H=2048, E=64, k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group="top2", renorm=True, scale=2.5),
        dict(name="linear_token", op="linear", T=1, N=2048, K=2048, type="fp16", act="none", bias=False, res=True),
        dict(name="linear_batch", op="linear", T=32, N=5632, K=2048, type="e4m3", act="silu", bias=False, res=False),
        dict(name="linear_ragged", op="linear", T=1333, N=2817, K=2064, type="fp16", act="gelu", bias=True, res=True),
        dict(name="linear_prompt", op="linear", T=8192, N=5632, K=4096, type="e4m3", act="silu", bias=True,
             res=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "linear"])
    if op == "norm":
        H = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            H = (H + 127) // 128 * 128
        T = _log(rng, 1, min(16384, 8192 * 4096 // H))
        fp16, e4m3 = rng.choice([(True, False), (False, True), (True, True)])
        return dict(op="norm", T=T, H=H, add=rng.random() < 0.7, fp16=fp16, e4m3=e4m3)
    if op == "route":
        E = rng.choice([8, 16, 24, 32, 33, 48, 60, 64])
        H = 128 * rng.randint(1, 32)
        T = _log(rng, 1, min(16384, 4096 * 2048 * 64 // (H * E)))
        n_group = rng.choice([g for g in (1, 1, 2, 3, 4, 8) if E % g == 0])
        topk_group = rng.randint(1, n_group)
        k = rng.randint(1, min(8, topk_group * (E // n_group)))
        group = "top2" if E // n_group >= 2 and rng.random() < 0.5 else "max"
        return dict(op="route", T=T, H=H, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, n_group=n_group, topk_group=topk_group, group=group,
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
    N, K = _log(rng, 64, 8192), 16 * _log(rng, 8, 512)
    if rng.random() < 0.6:
        N = (N + 127) // 128 * 128
    T = _log(rng, 1, max(1, min(16384, 8192 * 5632 * 4096 // (N * K))))
    return dict(op="linear", T=T, N=N, K=K, type=rng.choice(["fp16", "e4m3"]),
                act=rng.choice(["none", "silu", "gelu", "gelu_tanh"]), bias=rng.random() < 0.5,
                res=rng.random() < 0.5)


def work(case):
    T = case["T"]
    if case["op"] == "norm":
        n = T * case["H"]
        by = 2 * n * (1 + (2 if case["add"] else 0) + (1 if case["fp16"] else 0)) + (n + 4 * T if case["e4m3"] else 0)
        return {"bytes": by + 2 * case["H"], "flops": 6 * n}
    if case["op"] == "route":
        H, E, k = case["H"], case["E"], case["k"]
        return {"bytes": 2 * T * H + 2 * H * E + 4 * T * E + 16 * T * k + 8 * E + 8, "flops": 2 * T * H * E}
    N, K = case["N"], case["K"]
    size = 2 if case["type"] == "fp16" else 1
    by = size * (T * K + N * K) + 2 * T * N * (2 if case["res"] else 1) + (4 * N if case["bias"] else 0)
    return {"bytes": by + (4 * (T + N) if size == 1 else 0), "flops": 2 * T * N * K}


def _quantise(a):
    """Rows of `a` in e4m3 with one FP32 scale a row."""
    s = a.abs().amax(dim=1).clamp_min(1e-12) / E4M3_MAX
    return (a / s[:, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2654435761 % (1 << 31) + 17)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)

    T = case["T"]
    s = {"case": case}
    if case["op"] == "norm":
        H = case["H"]
        # a residual stream: channels of very different sizes, one layer's output beside it
        gain = torch.exp(randn(H))
        s["x"] = (randn(T, H) * gain).half()
        s["y"] = (randn(T, H) * 0.5).half() if case["add"] else None
        s["w"] = (1.0 + 0.2 * randn(H)).half()
        s["sum"] = torch.empty_like(s["x"]) if case["add"] else None
        s["norm"] = torch.empty_like(s["x"]) if case["fp16"] else None
        s["q"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV) if case["e4m3"] else None
        s["q_scale"] = torch.empty(T, dtype=torch.float32, device=DEV) if case["e4m3"] else None
        return s
    if case["op"] == "route":
        H, E, k = case["H"], case["E"], case["k"]
        s["x"] = randn(T, H).half()
        s["wr"] = (randn(H, E) / math.sqrt(H)).half()
        s["bias"] = 0.05 * randn(E) if case["bias"] else None

        def i32(*shape):
            return torch.empty(shape, dtype=torch.int32, device=DEV)

        s["logits"] = torch.empty((T, E), dtype=torch.float32, device=DEV)
        s["topk_w"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
        s["topk_ids"], s["expert_offsets"] = i32(T, k), i32(E + 1)
        s["sorted_pairs"], s["pair_pos"], s["active_list"], s["n_active"] = i32(T * k), i32(T * k), i32(E), i32(1)
        return s
    N, K = case["N"], case["K"]
    x, w = randn(T, K), randn(N, K) / math.sqrt(K)
    s["x_scale"] = s["w_scale"] = None
    if case["type"] == "fp16":
        s["x"], s["w"] = x.half(), w.half()
    else:
        (s["x"], s["x_scale"]), (s["w"], s["w_scale"]) = _quantise(x), _quantise(w)
    s["bias"] = 0.1 * randn(N) if case["bias"] else None
    s["res"] = randn(T, N).half() if case["res"] else None
    s["y"] = torch.empty((T, N), dtype=torch.float16, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _norm_plain(s):
    x, y, w = s["x"], s["y"], s["w"]
    v = x if y is None else (x.float() + y.float()).half()   # the FP32 sum of two FP16 values rounds like the exact one
    ms = v.double().square().mean(dim=1, keepdim=True)       # in 64 bits: the 8-bit rounding borders
    r = (1.0 / torch.sqrt(ms + _eps64())).float()
    n = v.float() * r * w.float()
    out = {}
    if y is not None:
        out["sum"] = v
    if s["norm"] is not None:
        out["norm"] = n.half()
    if s["q"] is not None:
        a = n.abs().amax(dim=1).clamp_min(AMAX_FLOOR)
        out["q_scale"] = a / _c32(E4M3_MAX)
        out["q"] = (n * (_c32(E4M3_MAX) / a)[:, None]).to(torch.float8_e4m3fn)
    return out


def _c32(v):
    return torch.full((), v, dtype=torch.float32, device=DEV)


def _eps64():
    return float(np.float32(EPS))


def _route_plain(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    # logits: products of FP16 values summed in 64 bits and rounded once (selection borders)
    logits = (s["x"].double() @ s["wr"].double()).float()
    l = logits.double()
    if c["score"] == "softmax":
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        score = e / e.sum(dim=1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    choice = score if s["bias"] is None else score + s["bias"].double()
    low = torch.full((), -math.inf, dtype=torch.float64, device=DEV)
    choice = torch.where(torch.isnan(choice), low, choice)
    if G > 1:
        by = choice.view(T, G, E // G)
        best = by.amax(dim=2) if c["group"] == "max" else torch.sort(by, dim=2, descending=True).values[:, :, :2].sum(2)
        rank = torch.sort(best, dim=1, descending=True, stable=True).indices
        kept = torch.zeros((T, G), dtype=torch.bool, device=DEV)
        kept.scatter_(1, rank[:, :c["topk_group"]], True)
        choice = torch.where(kept.repeat_interleave(E // G, dim=1), choice, low)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(score, 1, ids)
    if c["renorm"]:
        den = w.sum(dim=1, keepdim=True)
        w = torch.where(den > 0, w / den, torch.zeros_like(w))
    w = (w * c["scale"]).float()
    flat = ids.reshape(-1)
    pairs = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(pairs)
    pos[pairs] = torch.arange(T * k, device=DEV)
    counts = (flat[:, None] == torch.arange(E, device=DEV)[None, :]).sum(dim=0)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    none = torch.full((E,), E, dtype=torch.int64, device=DEV)
    active = torch.sort(torch.where(counts > 0, torch.arange(E, device=DEV), none)).values
    active = torch.where(active < E, active, torch.full_like(active, -1))
    whole = dict(topk_ids=ids, expert_offsets=offsets, sorted_pairs=pairs, pair_pos=pos, active_list=active,
                 n_active=(counts > 0).sum().reshape(1))
    return {"logits": logits, "topk_w": w, **{name: v.to(torch.int32) for name, v in whole.items()}}


def _linear_plain(s):
    c = s["case"]
    acc = s["x"].float() @ s["w"].float().t()
    if s["x_scale"] is not None:
        acc = acc * (s["x_scale"][:, None] * s["w_scale"][None, :])
    if s["bias"] is not None:
        acc = acc + s["bias"][None, :]
    if c["act"] == "silu":
        acc = acc / (1.0 + torch.exp(-acc))
    elif c["act"] == "gelu":
        acc = 0.5 * acc * (1.0 + torch.erf(acc * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        acc = 0.5 * acc * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (acc + 0.044715 * acc * acc * acc)))
    if s["res"] is not None:
        acc = acc + s["res"].float()
    return acc.half()


# ------------------------------------------------------------------ the library's calls
def _norm_own(s):
    from w4a16_routed_expert_amd import binding as B
    T, H = s["x"].shape
    B.moe_residual_rmsnorm(s["x"], s["y"], s["w"], EPS, T, H, sum_out=s["sum"], norm=s["norm"], q=s["q"],
                           q_scale=s["q_scale"])
    return {name: s[name] for name in ("sum", "norm", "q", "q_scale") if s[name] is not None}


def _route_own(s):
    from w4a16_routed_expert_amd import binding as B
    c = s["case"]
    if "ws" not in s:      # kept by the program: zero-filled once, the rule made once
        s["ws"] = torch.zeros(B.moe_route_scored_workspace_size(c["T"], c["H"], c["E"]), dtype=torch.uint8, device=DEV)
        s["rule"] = B.route_rule(score=B.MOE_SCORE_SOFTMAX if c["score"] == "softmax" else B.MOE_SCORE_SIGMOID,
                                 n_group=c["n_group"], topk_group=c["topk_group"],
                                 group_score=B.MOE_GROUP_MAX if c["group"] == "max" else B.MOE_GROUP_TOP2,
                                 renormalize=c["renorm"], scale=c["scale"])
    B.moe_route_scored(s["x"], s["wr"], s["bias"], c["T"], c["H"], c["E"], c["k"], s["rule"], s["logits"],
                       s["topk_ids"], s["topk_w"], s["expert_offsets"], s["sorted_pairs"], s["pair_pos"],
                       s["active_list"], s["n_active"], s["ws"], s["ws"].numel())
    return {name: s[name] for name in ("logits", "topk_w", "topk_ids", "expert_offsets", "sorted_pairs", "pair_pos",
                                       "active_list", "n_active")}


def _linear_own(s):
    from w4a16_routed_expert_amd import binding as B
    c = s["case"]
    if "ws" not in s:
        s["type"] = B.MOE_LINEAR_FP16 if c["type"] == "fp16" else B.MOE_LINEAR_E4M3
        s["act"] = {"none": B.MOE_ACT_NONE, "silu": B.MOE_ACT_SILU, "gelu": B.MOE_ACT_GELU,
                    "gelu_tanh": B.MOE_ACT_GELU_TANH}[c["act"]]
        s["ws"] = torch.empty(B.moe_linear_workspace_size(c["T"], c["N"], c["K"], s["type"]), dtype=torch.uint8,
                              device=DEV)
    B.moe_linear(s["x"], s["w"], c["T"], c["N"], c["K"], s["type"], s["y"], x_scale=s["x_scale"],
                 w_scale=s["w_scale"], bias=s["bias"], act=s["act"], residual=s["res"], ws=s["ws"],
                 ws_bytes=s["ws"].numel())
    return s["y"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _norm_own, "route": _route_own, "linear": _linear_own}[op](state)
    return {"norm": _norm_plain, "route": _route_plain, "linear": _linear_plain}[op](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        f = {name: s[name].cpu().numpy().astype(np.float64) for name in ("x", "y", "w") if s[name] is not None}
        out, v = {}, f["x"]
        if case["add"]:
            v = np.asarray(f["x"] + f["y"], dtype=np.float64)
            out["sum"] = v
            v = v.astype(np.float16).astype(np.float64)      # the stream is FP16: the norm reads the rounded sum
        n = v * f["w"][None, :] / np.sqrt(np.einsum("th,th->t", v, v)[:, None] / case["H"] + _eps64())
        if case["fp16"]:
            out["norm"] = n
        if case["e4m3"]:
            scale = np.maximum(np.max(np.abs(n), axis=1), AMAX_FLOOR) / E4M3_MAX
            out["q_scale"] = scale
            z = np.abs(n) / scale[:, None]
            # nearest e4m3 value: a step of 2^-3 of the value's power of two, at least 2^-9
            step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(z, 2.0 ** -20))), -6.0) - 3.0)
            out["q"] = np.copysign(np.rint(z / step) * step, n)
        return out
    if case["op"] == "route":
        T, E, k, G = case["T"], case["E"], case["k"], case["n_group"]
        x, wr = (s[name].cpu().numpy().astype(np.float64) for name in ("x", "wr"))
        l = np.matmul(x, wr)
        r = l.astype(np.float32).astype(np.float64)          # the definition's logit is the FP32 value
        if case["score"] == "softmax":
            score = np.exp(r - r.max(axis=1)[:, None])
            score /= score.sum(axis=1)[:, None]
        else:
            score = np.reciprocal(1.0 + np.exp(-r))
        c = score + (0.0 if s["bias"] is None else s["bias"].cpu().numpy().astype(np.float64)[None, :])
        in_group = np.arange(E) // (E // G)
        if G > 1:
            parts = np.sort(c.reshape(T, G, E // G), axis=2)
            value = parts[:, :, -1] if case["group"] == "max" else parts[:, :, -1] + parts[:, :, -2]
            place = np.argsort(np.argsort(-value, axis=1, kind="stable"), axis=1)
            c = np.where(place[:, in_group] < case["topk_group"], c, -np.inf)
        ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
        w = np.take_along_axis(score, ids, axis=1)
        if case["renorm"]:
            w = w / w.sum(axis=1)[:, None]
        return {"logits": l, "topk_w": w * case["scale"], "topk_ids": None, "expert_offsets": None,
                "sorted_pairs": None, "pair_pos": None, "active_list": None, "n_active": None}
    rows = max(1, (1 << 25) // max(case["N"], case["K"]))    # chunks of tokens: bounded memory
    w = s["w"].to(torch.float64)
    if s["w_scale"] is not None:
        w = w * s["w_scale"].to(torch.float64).unsqueeze(1)
    w = w.t().contiguous()
    parts = []
    for t0 in range(0, case["T"], rows):
        x = s["x"][t0:t0 + rows].to(torch.float64)
        if s["x_scale"] is not None:
            x = x * s["x_scale"][t0:t0 + rows].to(torch.float64).unsqueeze(1)
        z = torch.mm(x, w)
        if case["bias"]:
            z += s["bias"].to(torch.float64)
        if case["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        elif case["act"] == "gelu_tanh":
            z = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
        if case["res"]:
            z += s["res"][t0:t0 + rows].to(torch.float64)
        parts.append(z)
    return torch.cat(parts)
