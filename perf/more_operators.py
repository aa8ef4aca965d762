"""What a mixture-of-experts block computes around dispatch and combine, and in place of them for a few tokens, as cases to measure.

Kinds of a case:

  gate        gate_topk: router logits -> the top-k experts of every token and their weights
  gate_bwd    gate_topk_backward: gradient of the logits from that of the weights
  linear      linear: bf16 rows times a weight, with bias, activation and residual in the epilogue
  linear_bwd  linear_backward: gradients of its rows, its weight and its bias
  layer       expert_layer / expert_layer_fp8: a few tokens through all of their experts and back, bf16 or E4M3 weights

``own`` False: elementary torch operations; True: this package's entry points.
"""
import math

import numpy as np
import torch

own = False

FP8 = torch.float8_e4m3fn


def listed():
    return [
        # prefill or training: 16384 tokens, selection by biased scores among the best 4 of 8 groups of 32 experts
        dict(name="gate_prefill_grouped", kind="gate", N=16384, E=256, K=8, score="sigmoid", bias=True, groups=8, top_groups=4, renorm=True,
             scale=2.5, dtype="f32", masked=False),
        # decoding: a small batch over 64 experts, some of them switched off; latency
        dict(name="gate_decode", kind="gate", N=32, E=64, K=6, score="softmax", bias=False, groups=1, top_groups=1, renorm=True, scale=1.0,
             dtype="bf16", masked=True),
        # training: the dense gradient of a softmax over 256 experts
        dict(name="gate_bwd_softmax", kind="gate_bwd", N=16384, E=256, K=8, score="softmax", renorm=False, scale=1.0, dtype="f32"),
        # training: the sparse gradient of renormalised sigmoid scores, 160 experts
        dict(name="gate_bwd_sigmoid", kind="gate_bwd", N=4096, E=160, K=6, score="sigmoid", renorm=True, scale=2.5, dtype="bf16"),
        # the router's own product: 4096 tokens' fp32 logits over 256 experts
        dict(name="linear_router", kind="linear", M=4096, N=256, K=7168, act="none", bias=False, residual=False, out="f32", save=False),
        # decoding: first product of a shared expert, 16 tokens; reading the weight is what it costs
        dict(name="linear_decode_swiglu", kind="linear", M=16, N=4096, K=7168, act="swiglu", bias=False, residual=False, out="bf16", save=False),
        # training: the same for 8192 tokens, the values before the activation kept for the backward pass
        dict(name="linear_train_swiglu", kind="linear", M=8192, N=4096, K=7168, act="swiglu", bias=False, residual=False, out="bf16", save=True),
        # a ragged prompt: a biased product, its activation, and the residual stream added
        dict(name="linear_prompt_gelu", kind="linear", M=1003, N=7168, K=2048, act="gelu", bias=True, residual=True, out="bf16", save=False),
        # training: backward of a shared expert's first product
        dict(name="linear_bwd_swiglu", kind="linear_bwd", M=4096, N=4096, K=7168, act="swiglu", bias=False),
        # training on a ragged batch: backward through gelu and bias
        dict(name="linear_bwd_gelu", kind="linear_bwd", M=777, N=4096, K=1024, act="gelu", bias=True),
        # decoding one token on one GPU: eight experts of 88 MB each
        dict(name="layer_one_token", kind="layer", N=1, K=8, E=32, experts=32, H=7168, I=2048, fp8=False, residual=True),
        # decoding 64 tokens on one of four ranks: 64 of 256 experts are here, weights in E4M3
        dict(name="layer_fp8_64_tokens", kind="layer", N=64, K=8, E=64, experts=256, H=7168, I=2048, fp8=True, residual=False),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(v) // step * step)


def draw(rng):
    kind = rng.choice(["gate", "gate", "gate_bwd", "linear", "linear", "linear", "linear_bwd", "layer", "layer", "layer"])
    if kind in ("gate", "gate_bwd"):
        c = dict(kind=kind, N=_log(rng, 1, 16384), E=_log(rng, 8, 384), K=0, score=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]))
        c["K"] = rng.randint(1, min(8, c["E"]))
        if kind == "gate":
            c["bias"], c["masked"] = rng.random() < 0.5, rng.random() < 0.3
            c["groups"] = rng.choice([1, 1, 4, 8])
            c["E"] = c["E"] // (2 * c["groups"]) * 2 * c["groups"] or 2 * c["groups"]
            c["top_groups"] = rng.randint(1, c["groups"])
            c["K"] = min(c["K"], c["E"] // c["groups"] * c["top_groups"])
        return c
    if kind.startswith("linear"):
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
        c = dict(kind=kind, M=_log(rng, 1, 8192 if kind == "linear" else 4096), N=_log(rng, 16, 4096, 16), K=_log(rng, 64, 7168, 8), act=act,
                 bias=rng.random() < 0.5)
        if kind == "linear":
            c["residual"], c["out"], c["save"] = rng.random() < 0.5, rng.choice(["bf16", "bf16", "f32"]), act != "none" and rng.random() < 0.4
        return c
    fp8 = rng.random() < 0.5
    E = rng.choice([4, 8, 16, 32, 64])
    c = dict(kind=kind, N=_log(rng, 1, 64), K=rng.randint(1, 8), E=E, experts=E * rng.choice([1, 1, 2, 4]), H=_log(rng, 256, 7168, 128 if fp8 else 8),
             I=_log(rng, 128, 2048, 128 if fp8 else 8), fp8=fp8, residual=rng.random() < 0.5)
    c["K"] = min(c["K"], c["experts"])
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed, device="cpu"):
    return torch.Generator(device=device).manual_seed(1000003 * int(seed) + 11)


def _randn(shape, gd, std=1.0):
    return torch.randn(shape, generator=gd, device="cuda", dtype=torch.float32).mul_(std)


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _quant_blocks(w):
    """E4M3 codes of w [E, N, K] with a scale for each 128 x 128 block."""
    E, N, K = w.shape
    v = w.view(E, N // 128, 128, K // 128, 128)
    s = v.abs().amax((2, 4)).clamp_min(1e-4) / 448.0
    return (v / s.view(E, N // 128, 1, K // 128, 1)).to(FP8).view(E, N, K), s


def prepare(case, seed):
    c, gd = case, _gen(seed, "cuda")
    s, kind = dict(case=c), case["kind"]
    dev = dict(device="cuda")
    if kind in ("gate", "gate_bwd"):
        N, E, K = c["N"], c["E"], c["K"]
        logits = _randn((N, E), gd, 1.5)
        s["idx"] = torch.zeros((N, K), dtype=torch.int64, **dev)
        if kind == "gate":
            if c["masked"]:  # a quarter of the experts switched off, and one token that takes no part
                off = torch.rand((E,), generator=gd, **dev) < 0.25
                logits = logits.masked_fill_(off.unsqueeze(0), float("-inf"))
                logits[N // 2] = float("-inf")
            s["bias"] = _randn((E,), gd, 0.1) if c["bias"] else None
            s["weights"] = torch.zeros((N, K), dtype=torch.float32, **dev)
        else:
            s["idx"] = torch.rand((N, E), generator=gd, **dev).topk(K, dim=1).indices
            s["dw"] = _randn((N, K), gd)
            s["dlogits"] = torch.zeros((N, E), dtype=_dtype(c["dtype"]), **dev)
        s["logits"] = logits.to(_dtype(c["dtype"]))
        return s
    if kind.startswith("linear"):
        M, N, K = c["M"], c["N"], c["K"]
        out = N // 2 if c["act"] == "swiglu" else N
        s["x"] = _randn((M, K), gd).to(torch.bfloat16)
        s["w"] = _randn((N, K), gd, K ** -0.5).to(torch.bfloat16)
        s["bias"] = _randn((N,), gd, 0.5) if c["bias"] else None
        if kind == "linear":
            s["residual"] = _randn((M, out), gd).to(torch.bfloat16) if c["residual"] else None
            s["y"] = torch.zeros((M, out), dtype=_dtype(c["out"]), **dev)
            s["z"] = torch.zeros((M, N), dtype=torch.bfloat16, **dev) if c["save"] else None
            return s
        s["z"] = _randn((M, N), gd).to(torch.bfloat16) if c["act"] != "none" else None
        s["dy"] = _randn((M, out), gd).to(torch.bfloat16)
        s["dx"] = torch.zeros((M, K), dtype=torch.bfloat16, **dev)
        s["dweight"] = torch.zeros((N, K), dtype=torch.bfloat16, **dev)
        s["dbias"] = torch.zeros((N,), dtype=torch.float32, **dev) if c["bias"] else None
        s["dz"] = torch.zeros((M, N), dtype=torch.bfloat16, **dev)
        s["workspace"] = torch.zeros((min(256, -(-M // 16)), N), dtype=torch.float32, **dev)
        return s
    N, K, E, H, I = c["N"], c["K"], c["E"], c["H"], c["I"]
    s["first"] = c["experts"] // E // 2 * E  # a rank in the middle
    s["idx"] = torch.rand((N, c["experts"]), generator=gd, **dev).topk(K, dim=1).indices
    s["weights"] = torch.softmax(_randn((N, K), gd), 1)
    s["x"] = _randn((N, H), gd).to(torch.bfloat16)
    s["residual"] = _randn((N, H), gd).to(torch.bfloat16) if c["residual"] else None
    s["y"] = torch.zeros((N, H), dtype=torch.bfloat16, **dev)
    s["workspace"] = torch.zeros((N * K, I), dtype=torch.bfloat16, **dev)
    w1, w2 = _randn((E, 2 * I, H), gd, H ** -0.5), None
    if c["fp8"]:
        s["w1"], s["w1_scales"] = _quant_blocks(w1)
    else:
        s["w1"] = w1.to(torch.bfloat16)
    del w1
    w2 = _randn((E, H, I), gd, 2 * I ** -0.5)
    if c["fp8"]:
        s["w2"], s["w2_scales"] = _quant_blocks(w2)
    else:
        s["w2"] = w2.to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ plain forms
def _scores(l, score):
    """Scores of logits l (masked ones are -inf): they add to one, or each stands for itself."""
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    return e / e.sum(1, keepdim=True).clamp_min(1e-30)


def _first_best(v, k):
    """Places of the k largest values of each row, the largest first, equal ones by their place."""
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :k]


def _gate(s):
    c = s["case"]
    N, E, K = c["N"], c["E"], c["K"]
    l = s["logits"].double()  # two scores next to each other choose another expert: 64 bits decide
    off = torch.isinf(l)
    pick = l
    if s["bias"] is not None or c["groups"] > 1:
        pick = _scores(l, c["score"])
        pick = (pick if s["bias"] is None else pick + s["bias"].double()).masked_fill(off, float("-inf"))
    if c["groups"] > 1:
        best = pick.view(N, c["groups"], -1).sort(2, descending=True).values[:, :, :2].sum(2)
        inside = torch.zeros((N, c["groups"]), dtype=torch.bool, device="cuda").scatter_(1, _first_best(best, c["top_groups"]), True)
        pick = pick.masked_fill(~inside.repeat_interleave(E // c["groups"], 1), float("-inf"))
    idx = _first_best(pick, K)
    none = torch.isinf(pick.gather(1, idx))
    w = _scores(s["logits"].float(), c["score"]).gather(1, idx).masked_fill(none, 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-30)
    return idx.masked_fill(none, -1), w * c["scale"]


def _gate_backward(s):
    c = s["case"]
    p = _scores(s["logits"].float(), c["score"])
    own_p, dw = p.gather(1, s["idx"]), s["dw"] * c["scale"]
    if c["renorm"]:  # weights = p / sum of the chosen p
        total = own_p.sum(1, keepdim=True)
        dw = (dw - (dw * own_p).sum(1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter_(1, s["idx"], dw)
    d = dp * p * (1.0 - p) if c["score"] == "sigmoid" else p * (dp - (dp * p).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    if act == "swiglu":
        g, u = z.chunk(2, 1)
        return g / (1.0 + torch.exp(-g)) * u
    return z


def _act_backward(z, dy, act):
    if act == "relu":
        return dy * (z > 0)
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        return dy * sig * (1.0 + z * (1.0 - sig))
    if act == "gelu":
        return dy * (0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5)
    if act == "gelu_tanh":
        r = (2 / math.pi) ** 0.5
        t = torch.tanh(r * (z + 0.044715 * z * z * z))
        return dy * (0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * r * (1.0 + 3 * 0.044715 * z * z))
    if act == "swiglu":
        g, u = z.chunk(2, 1)
        sig = 1.0 / (1.0 + torch.exp(-g))
        return torch.cat([dy * u * sig * (1.0 + g * (1.0 - sig)), dy * g * sig], 1)
    return dy


def _linear(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    z = z if s["bias"] is None else z + s["bias"]
    y = _act(z, c["act"])
    y = (y if s["residual"] is None else y + s["residual"].float()).to(_dtype(c["out"]))
    return (y, z.to(torch.bfloat16)) if c["save"] else y


def _linear_backward(s):
    c = s["case"]
    dz = s["dy"].float() if c["act"] == "none" else _act_backward(s["z"].float(), s["dy"].float(), c["act"])
    out = (dz @ s["w"].float()).to(torch.bfloat16), (dz.t() @ s["x"].float()).to(torch.bfloat16)
    return (*out, dz.sum(0)) if c["bias"] else out


def _floats(s, name, at=None):
    """Weights in fp32: of the experts `at`, or of all."""
    w = s[name] if at is None else s[name].view(torch.uint8)[at].view(FP8) if s["case"]["fp8"] else s[name][at]
    if not s["case"]["fp8"]:
        return w.float()
    sc = s[name + "_scales"] if at is None else s[name + "_scales"][at]
    E, N, K = w.shape
    return (w.float().view(E, N // 128, 128, K // 128, 128) * sc.view(E, N // 128, 1, K // 128, 1)).view(E, N, K)


def _layer(s):
    c = s["case"]
    N, K, E, I = c["N"], c["K"], c["E"], c["I"]
    e = s["idx"] - s["first"]
    here = (e >= 0) & (e < E)
    if N * K <= E:  # every entry with its expert's weights
        at, x = torch.where(here, e, 0).view(-1), s["x"].float().repeat_interleave(K, 0).unsqueeze(2)
        h = torch.bmm(_floats(s, "w1", at), x).squeeze(2)
        a = h[:, :I] / (1.0 + torch.exp(-h[:, :I])) * h[:, I:]
        z = torch.bmm(_floats(s, "w2", at), a.unsqueeze(2)).view(N, K, -1)
        y = (z * torch.where(here, s["weights"], 0.0).unsqueeze(2)).sum(1)
    else:  # every expert on all tokens
        gate = torch.zeros((N, E + 1), device="cuda").scatter_add_(1, torch.where(here, e, E), s["weights"])[:, :E]
        h = torch.matmul(s["x"].float(), _floats(s, "w1").transpose(1, 2))
        a = h[:, :, :I] / (1.0 + torch.exp(-h[:, :, :I])) * h[:, :, I:]
        a = a * gate.t().unsqueeze(2)
        y = torch.bmm(a, _floats(s, "w2").transpose(1, 2)).sum(0)
    return (y if s["residual"] is None else y + s["residual"].float()).to(torch.bfloat16)


def _plain(s):
    form = dict(gate=_gate, gate_bwd=_gate_backward, linear=_linear, linear_bwd=_linear_backward, layer=_layer)
    return form[s["case"]["kind"]](s)


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import combine_get_dispatch_histogram_amd as miep
    c, kind = s["case"], s["case"]["kind"]
    if kind == "gate":
        miep.gate_topk_into(s["logits"], s["idx"], s["weights"], score=c["score"], bias=s["bias"], num_groups=c["groups"],
                            topk_groups=c["top_groups"], renormalize=c["renorm"], scale=c["scale"])
        return s["idx"], s["weights"]
    if kind == "gate_bwd":
        miep.gate_topk_backward_into(s["dw"], s["logits"], s["idx"], s["dlogits"], score=c["score"], renormalize=c["renorm"], scale=c["scale"])
        return s["dlogits"]
    act = None if c.get("act") == "none" else c.get("act")
    if kind == "linear":
        miep.linear_into(s["x"], s["w"], s["y"], bias=s["bias"], activation=act, residual=s["residual"], z=s["z"])
        return (s["y"], s["z"]) if c["save"] else s["y"]
    if kind == "linear_bwd":
        miep.linear_backward_into(s["dy"], s["x"], s["w"], activation=act, z=s["z"], dx=s["dx"], dw=s["dweight"], dbias=s["dbias"],
                                  dz=s["dz"], workspace=s["workspace"])
        return (s["dx"], s["dweight"], s["dbias"]) if c["bias"] else (s["dx"], s["dweight"])
    if c["fp8"]:
        miep.expert_layer_fp8_into(s["x"], s["idx"], s["weights"], s["w1"], s["w1_scales"], s["w2"], s["w2_scales"], s["y"], s["workspace"],
                                   first_expert=s["first"], residual=s["residual"])
    else:
        miep.expert_layer_into(s["x"], s["idx"], s["weights"], s["w1"], s["w2"], s["y"], s["workspace"], first_expert=s["first"],
                               residual=s["residual"])
    return s["y"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def work(case):
    c, kind = case, case["kind"]
    if kind in ("gate", "gate_bwd"):
        b = 4 if c["dtype"] == "f32" else 2
        if kind == "gate":
            return dict(bytes=c["N"] * (c["E"] * b + c["K"] * 12) + (4 * c["E"] if c["bias"] else 0), flops=10 * c["N"] * c["E"])
        read = c["E"] if c["score"] == "softmax" and not c["renorm"] else c["K"]  # a renormalised weight depends on the chosen logits alone
        return dict(bytes=c["N"] * (b * (read + c["E"]) + c["K"] * 12), flops=10 * c["N"] * read)
    if kind.startswith("linear"):
        M, N, K = c["M"], c["N"], c["K"]
        out = N // 2 if c["act"] == "swiglu" else N
        if kind == "linear":
            each = (4 if c["out"] == "f32" else 2) + (2 if c["residual"] else 0)
            return dict(bytes=2 * (M + N) * K + M * out * each + (2 * M * N if c["save"] else 0) + (4 * N if c["bias"] else 0), flops=2 * M * N * K)
        return dict(bytes=2 * M * (out + 2 * K) + (2 * M * N if c["act"] != "none" else 0) + 4 * N * K + (4 * N if c["bias"] else 0), flops=4 * M * N * K)
    entries = c["N"] * c["K"] * c["E"] / c["experts"]
    live = c["E"] * (1 - (1 - c["K"] / c["experts"]) ** c["N"])  # experts that some token chose, about
    b = 1 if c["fp8"] else 2
    return dict(bytes=3 * live * c["I"] * c["H"] * b + 2 * c["N"] * c["H"] * (3 if c["residual"] else 2) + 12 * c["N"] * c["K"],
                flops=6 * entries * c["I"] * c["H"])


# ------------------------------------------------------------------ 64 bits
def _log_scores(l, score):
    """Logarithms of the scores in 64 bits."""
    if score == "sigmoid":
        return torch.minimum(l, torch.zeros_like(l)) - torch.log1p(torch.exp(-l.abs()))
    return l - torch.logsumexp(l, 1, keepdim=True)


def _best_experts(l, bias, c):
    """The chosen experts of every token (-1: none left) on the host."""
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        if bias is None and c["groups"] == 1:
            v = l
        elif c["score"] == "sigmoid":
            v = 1 / (1 + np.exp(-l))
        else:
            e = np.exp(l - l.max(1, keepdims=True))
            v = e / e.sum(1, keepdims=True)
    v = v if bias is None else v + bias.astype(np.float64)
    v[np.isinf(l)] = -np.inf
    if c["groups"] > 1:
        rows, per = np.arange(len(v))[:, None], c["E"] // c["groups"]
        two = np.partition(v.reshape(len(v), c["groups"], per), per - 2, axis=2)[:, :, -2:].sum(2)
        left = np.ones(two.shape, dtype=bool)
        left[rows, np.argsort(-two, axis=1, kind="stable")[:, :c["top_groups"]]] = False
        v[np.repeat(left, per, axis=1)] = -np.inf
    idx = np.argsort(-v, axis=1, kind="stable")[:, :c["K"]]
    return np.where(np.isinf(np.take_along_axis(v, idx, 1)), -1, idx)


def exact(case, seed):
    s, c, kind = prepare(case, seed), case, case["kind"]
    if kind == "gate":
        idx = torch.from_numpy(_best_experts(s["logits"].double().cpu().numpy(), None if s["bias"] is None else s["bias"].cpu().numpy(), c)).cuda()
        none = idx < 0
        v = _log_scores(s["logits"].double(), c["score"]).gather(1, idx.clamp_min(0)).masked_fill(none, float("-inf"))
        if c["renorm"]:
            v = v - torch.logsumexp(v, 1, keepdim=True)
        return None, torch.exp(v).masked_fill(none, 0.0) * c["scale"]
    if kind == "gate_bwd":
        l = s["logits"].double().requires_grad_()
        v = _log_scores(l, c["score"]).gather(1, s["idx"])
        w = torch.exp(v - torch.logsumexp(v, 1, keepdim=True) if c["renorm"] else v) * c["scale"]
        return torch.autograd.grad((w * s["dw"].double()).sum(), l)[0]
    fun = dict(none=lambda z: z, relu=torch.relu, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu,
               gelu_tanh=lambda z: torch.nn.functional.gelu(z, approximate="tanh"),
               swiglu=lambda z: torch.nn.functional.silu(z[:, :z.shape[1] // 2]) * z[:, z.shape[1] // 2:])
    if kind == "linear":
        z = s["x"].double() @ s["w"].double().t()
        z = z if s["bias"] is None else z + s["bias"].double()
        y = fun[c["act"]](z)
        y = y if s["residual"] is None else y + s["residual"].double()
        return (y, z) if c["save"] else y
    if kind == "linear_bwd":
        dz = s["dy"].double()
        if c["act"] != "none":
            z = s["z"].double().requires_grad_()
            dz = torch.autograd.grad((fun[c["act"]](z) * dz).sum(), z)[0]
        out = dz @ s["w"].double(), dz.t().contiguous() @ s["x"].double()
        return (*out, dz.sum(0)) if c["bias"] else out
    y = torch.zeros((c["N"], c["H"]), dtype=torch.float64, device="cuda") if s["residual"] is None else s["residual"].double()
    for e in range(c["E"]):
        n, k = (s["idx"] == s["first"] + e).nonzero(as_tuple=True)
        if n.numel():
            w1, w2 = s["w1"][e].double(), s["w2"][e].double()
            if c["fp8"]:
                w1 = w1 * s["w1_scales"][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
                w2 = w2 * s["w2_scales"][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            a = fun["swiglu"](s["x"][n].double() @ w1.t())
            y.index_add_(0, n, (a @ w2.t()) * s["weights"][n, k, None].double())
    return y
