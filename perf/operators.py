"""The expert operators that stand between dispatch and combine, as cases to measure.

Kinds of a case:

  order       expert_order: received rows (each with its local top-k experts) -> slots in expert order
  reduce      expert_reduce: expert outputs in slot order -> received rows, gate-weighted
  reduce_bwd  its gradient: slots' gradients and the gate weights' gradients
  gemm        grouped_gemm: bf16 rows times their expert's [N, K] weight, rows optionally gathered by index
  dgrad       grouped_gemm_dgrad: gradient of the rows
  wgrad       grouped_gemm_wgrad: gradient of the weights (fp32)
  fp8         grouped_gemm_fp8: E4M3 rows (a scale per 128 channels) times E4M3 weights (a scale per 128 x 128 block)
  swiglu      swiglu / swiglu_fp8: silu(gate) * up, to bf16 or cast per 128 channels to E4M3
  swiglu_bwd  swiglu_backward

``own`` False: elementary torch operations in 32 bits; True: this package's entry points.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn


def listed():
    return [
        # routing of 16384 tokens, top-8 of 256 experts, received by 64 ranks
        dict(name="order_16k_tokens", kind="order", N=16384, K=8, E=256, R=64, align=1, routing="uniform"),
        # one rank's share of 4096 tokens x top-8 over 8 ranks, combined back to its received rows
        dict(name="reduce_4k_tokens", kind="reduce", N=4096, K=8, E=32, R=1, H=7168, align=1, routing="masked"),
        # its gradient, on skewed routing
        dict(name="reduce_bwd_skewed", kind="reduce_bwd", N=4096, K=8, E=32, R=1, H=7168, align=1, routing="zipf"),
        # decoding: 8 local experts behind the low-latency dispatch, a few rows each: latency and weight reading
        dict(name="gemm_decode", kind="gemm", G=8, rows=29, cap=256, N=4096, K=7168, layout="slots", dist="even", gather=False),
        # training and prefill: one rank's 16384 expert rows, gathered from its received rows
        dict(name="gemm_train_gather", kind="gemm", G=32, rows=16384, cap=0, N=4096, K=7168, layout="ragged", dist="zipf", gather=True),
        # backward of the second product over ragged groups
        dict(name="dgrad_ragged", kind="dgrad", G=32, rows=8192, cap=0, N=7168, K=2048, layout="ragged", dist="zipf", gather=False),
        dict(name="wgrad_ragged", kind="wgrad", G=32, rows=8192, cap=0, N=7168, K=2048, layout="ragged", dist="zipf", gather=False),
        # low-latency FP8 serving: a handful of rows an expert
        dict(name="fp8_decode", kind="fp8", G=8, rows=61, cap=512, N=4096, K=7168, layout="slots", dist="even", gather=False, ue8m0=False),
        # low-latency FP8 serving of 32 x 128 tokens: about 128 rows an expert in 4096 slots
        dict(name="fp8_low_latency", kind="fp8", G=8, rows=1024, cap=4096, N=4096, K=7168, layout="slots", dist="even", gather=False, ue8m0=False),
        # FP8 prefill, second product, power-of-two scales
        dict(name="fp8_prefill_ue8m0", kind="fp8", G=32, rows=16384, cap=0, N=7168, K=2048, layout="ragged", dist="zipf", gather=False, ue8m0=True),
        # activation between the two FP8 products of the low-latency path
        dict(name="swiglu_fp8_low_latency", kind="swiglu", G=8, rows=1024, cap=4096, I=2048, layout="slots", dist="even", fp8=True),
        # activation's gradient in training
        dict(name="swiglu_bwd_train", kind="swiglu_bwd", G=32, rows=16384, cap=0, I=2048, layout="ragged", dist="zipf"),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(v) // step * step)


def draw(rng):
    kind = rng.choice(["order", "reduce", "reduce_bwd", "gemm", "gemm", "dgrad", "wgrad", "fp8", "fp8", "swiglu", "swiglu_bwd"])
    if kind in ("order", "reduce", "reduce_bwd"):
        R = rng.choice([1, 2, 4, 8]) if kind == "order" else rng.choice([1, 1, 2])
        c = dict(kind=kind, N=_log(rng, 16, 16384 if kind == "order" else 4096), K=rng.randint(1, 8), E=R * rng.choice([8, 16, 32]), R=R,
                 align=rng.choice([1, 1, 8, 128]), routing=rng.choice(["uniform", "zipf", "masked"]))
        if kind != "order":
            c["H"] = _log(rng, 128, 7168, 8)
        return c
    layout = rng.choice(["ragged", "slots"])
    G = rng.choice([1, 2, 5, 8, 16, 32])
    rows = _log(rng, 1, 8192)
    c = dict(kind=kind, G=G, rows=rows, cap=0, layout=layout, dist=rng.choice(["even", "zipf"]))
    if layout == "slots":
        c["dist"] = "even"
        c["cap"] = -(-rows // G) * 2 + rng.randint(0, 64)
    if kind.startswith("swiglu"):
        c["I"] = _log(rng, 128, 4096, 128 if kind == "swiglu" else 8)
        if kind == "swiglu":
            c["fp8"] = rng.random() < 0.5
        return c
    c["N"], c["K"] = _log(rng, 128, 4096, 8), _log(rng, 128, 7168, 128 if kind == "fp8" else 8)
    c["gather"] = kind in ("gemm", "wgrad", "fp8") and layout == "ragged" and rng.random() < 0.5
    if kind == "fp8":
        c["ue8m0"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed, device="cpu"):
    return torch.Generator(device=device).manual_seed(1000003 * int(seed) + 7)


def _groups(c, g):
    """Rows of every group and where they begin (host lists), and the rows of the whole layout."""
    G, rows = c["G"], c["rows"]
    if c["dist"] == "zipf":
        p = 1.0 / torch.arange(1, G + 1, dtype=torch.float64) ** 0.8
        p = p[torch.randperm(G, generator=g)]
        n = torch.bincount(torch.multinomial(p, rows, replacement=True, generator=g), minlength=G)
        if G > 4:  # an expert that no token chose
            few = int(n.argmin())
            n[int(n.argmax())] += n[few]
            n[few] = 0
    else:
        n = torch.bincount(torch.randint(0, G, (rows,), generator=g), minlength=G)
    if c["layout"] == "slots":
        n = n.clamp(max=c["cap"])
        begin = torch.arange(G) * c["cap"]
        total = G * c["cap"]
    else:
        begin = n.cumsum(0) - n
        total = int(n.sum())
    return n.tolist(), begin.tolist(), total


def _randn(shape, gd, std=1.0):
    return torch.randn(shape, generator=gd, device="cuda", dtype=torch.float32).mul_(std)


def _pow2_ceil(s):
    return torch.exp2(torch.ceil(torch.log2(s)))


def _quant_rows(x, ue8m0):
    v = x.view(x.shape[0], -1, 128)
    s = v.abs().amax(2).clamp_min(1e-4) / 448.0
    s = _pow2_ceil(s) if ue8m0 else s
    return (v / s.unsqueeze(2)).to(FP8).view(x.shape), s


def _quant_blocks(w, ue8m0):
    G, N, K = w.shape
    nb = -(-N // 128)
    if N % 128:
        w = torch.cat([w, w.new_zeros(G, nb * 128 - N, K)], 1)
    v = w.view(G, nb, 128, K // 128, 128)
    s = v.abs().amax((2, 4)).clamp_min(1e-4) / 448.0
    s = _pow2_ceil(s) if ue8m0 else s
    q = (v / s.view(G, nb, 1, K // 128, 1)).to(FP8).view(G, nb * 128, K)[:, :N].contiguous()
    return q, s


def _scale_arg(s, ue8m0):
    """Scales as a program holds them: fp32, or the exponent byte of each power of two."""
    return (torch.log2(s) + 127).round().to(torch.uint8) if ue8m0 else s


def _routing(c, g):
    """Received rows in a receive side of the worst case's size: their local top-k experts (-1 elsewhere, and behind the last row),
    gate weights and each rank's first row."""
    N, K, E, R = c["N"], c["K"], c["E"], c["R"]
    wide = E * 8 if c["routing"] == "masked" else E  # masked: seven eighths of the experts live elsewhere
    score = torch.rand((N, wide), generator=g)
    if c["routing"] == "zipf":
        score = torch.log(score) * torch.arange(1, wide + 1).float() ** 0.6
    idx = score.topk(K, dim=1).indices.cuda()
    wts = torch.softmax(torch.randn((N, K), generator=g), 1).cuda()
    L = E // R
    own_rank = torch.where(idx < E, idx // L, -1)
    member = (own_rank.unsqueeze(0) == torch.arange(R, device="cuda").view(R, 1, 1)).any(2)  # [R, N]
    at = member.nonzero()
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), member.sum(1).cumsum(0)])
    r, n = at[:, 0], at[:, 1]
    mine = own_rank[n] == r.unsqueeze(1)
    cap, rows = N * min(K, R), at.shape[0]
    local = torch.full((cap, K), -1, dtype=torch.int64, device="cuda")
    gate = torch.zeros((cap, K), device="cuda")
    local[:rows] = torch.where(mine, idx[n] - r.unsqueeze(1) * L, -1)
    gate[:rows] = torch.where(mine, wts[n], 0.0)
    return local, gate, off.to(torch.int32)


def prepare(case, seed):
    c, g, gd = case, _gen(seed), _gen(seed, "cuda")
    s = dict(case=c)
    kind = c["kind"]
    if kind in ("order", "reduce", "reduce_bwd"):
        s["topk"], s["weights"], s["offset"] = _routing(c, g)
        rows = s["topk"].shape[0]
        s["slots"] = rows * min(c["K"], c["E"] // c["R"]) + (c["align"] - 1) * c["E"]  # the most that can be needed
        dev = dict(dtype=torch.int32, device="cuda")
        s["begin"], s["count"] = torch.zeros(c["E"], **dev), torch.zeros(c["E"], **dev)
        s["slot_row"], s["row_slot"] = torch.zeros(s["slots"], **dev), torch.zeros((rows, c["K"]), **dev)
        s["workspace"] = torch.zeros((max(1, 256 // c["R"]), c["E"]), **dev)
        if kind != "order":
            begin, count, slot_row, row_slot = _order(s["topk"], s["offset"], c, s["slots"])
            s.update(begin=begin.int(), count=count.int(), slot_row=slot_row.int(), row_slot=row_slot.int())
            s["z"] = _randn((s["slots"], c["H"]), gd).to(torch.bfloat16)
            s["y"] = torch.zeros((rows, c["H"]), dtype=torch.bfloat16, device="cuda")
        if kind == "reduce_bwd":
            s["dy"] = _randn((rows, c["H"]), gd).to(torch.bfloat16)
            s["dz"] = torch.zeros_like(s["z"])
            s["dw"] = torch.zeros_like(s["weights"])
        return s
    n, begin, total = _groups(c, g)
    s["max_rows"], s["total"] = max(1, max(n)), total
    s["count"] = torch.tensor(n, dtype=torch.int32, device="cuda")
    s["begin"] = torch.tensor(begin, dtype=torch.int32, device="cuda")
    s["expected"] = -(-c["rows"] // c["G"])  # what a program knows of its batch: tokens x top-k over experts
    G = c["G"]
    if kind.startswith("swiglu"):
        I = c["I"]
        s["h"] = _randn((total, 2 * I), gd, 1.5).to(torch.bfloat16)
        if kind == "swiglu_bwd":
            s["da"] = _randn((total, I), gd).to(torch.bfloat16)
            s["dh"] = torch.zeros_like(s["h"])
        elif c["fp8"]:
            s["a"] = torch.zeros((total, I), dtype=torch.uint8, device="cuda").view(FP8)
            s["scales"] = torch.zeros((total, I // 128), dtype=torch.float32, device="cuda")
        else:
            s["a"] = torch.zeros((total, I), dtype=torch.bfloat16, device="cuda")
        return s
    N, K = c["N"], c["K"]
    src = total
    if c["gather"]:  # about two experts a received row
        src = max(1, total // 2)
        s["index"] = torch.randint(0, src, (total,), generator=gd, device="cuda", dtype=torch.int32)
    if kind != "wgrad":
        w = _randn((G, N, K), gd, K ** -0.5)
        if kind == "fp8":
            s["w"], ws = _quant_blocks(w, c["ue8m0"])
            s["w_scales"] = _scale_arg(ws, c["ue8m0"])
        else:
            s["w"] = w.to(torch.bfloat16)
        del w
    if kind in ("dgrad", "wgrad"):
        s["dy"] = _randn((total, N), gd).to(torch.bfloat16)
    if kind == "dgrad":
        s["dx"] = torch.zeros((total, K), dtype=torch.bfloat16, device="cuda")
        return s
    x = _randn((src, K), gd)
    if kind == "fp8":
        s["x"], xs = _quant_rows(x, c["ue8m0"])
        s["x_scales"] = _scale_arg(xs, c["ue8m0"])
    else:
        s["x"] = x.to(torch.bfloat16)
    if kind == "wgrad":
        s["dweight"] = torch.zeros((G, N, K), dtype=torch.float32, device="cuda")
    else:
        s["y"] = torch.zeros((total, N), dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _order(topk, offset, c, slots):
    """Stable order of the (row, k) entries by expert; padding and unused slots hold -1."""
    rows, K = topk.shape
    E, R, L = c["E"], c["R"], c["E"] // c["R"]
    row = torch.arange(rows, device=topk.device)
    rank = torch.searchsorted(offset.long(), row, right=True) - 1
    e = torch.where((topk >= 0) & (rank < R).unsqueeze(1), topk + (rank * L).unsqueeze(1), E).reshape(-1)
    by, at = torch.sort(e, stable=True)
    count = torch.zeros(E + 1, dtype=torch.int64, device=topk.device).scatter_add_(0, e, torch.ones_like(e))
    first = count.cumsum(0) - count
    padded = (count[:E] + c["align"] - 1) // c["align"] * c["align"]
    begin = padded.cumsum(0) - padded
    place = torch.cat([begin, begin.new_full((1,), slots)])[by] + torch.where(by < E, torch.arange(rows * K, device=topk.device) - first[by], 0)
    slot_row = torch.full((slots + 1,), -1, dtype=torch.int64, device=topk.device).scatter_(0, place, at // K)[:slots]
    row_slot = torch.empty_like(at).scatter_(0, at, torch.where(by < E, place, -1)).view(rows, K)
    return begin, count[:E], slot_row, row_slot


def _padded(s):
    """[G, max_rows] layout rows of every group, and which of them are rows."""
    i = torch.arange(s["max_rows"], device="cuda")
    live = i.unsqueeze(0) < s["count"].unsqueeze(1)
    return torch.where(live, s["begin"].long().unsqueeze(1) + i, s["total"]), live


def _live_rows(s):
    """[total, 1]: whether a layout row belongs to a group."""
    row = torch.arange(s["total"], device="cuda").unsqueeze(1)
    begin = s["begin"].long().unsqueeze(0)
    return ((row >= begin) & (row < begin + s["count"])).any(1, keepdim=True)


def _take(x, at, live):
    return x[torch.where(live, at, 0)].float().masked_fill_(~live.unsqueeze(2), 0.0)


def _put(at, v, total, dtype):
    out = torch.zeros((total + 1, v.shape[-1]), dtype=dtype, device="cuda")
    out[at.reshape(-1)] = v.reshape(-1, v.shape[-1]).to(dtype)
    return out[:total]


def _scales(s, t):
    return torch.exp2(t.float() - 127) if s["case"]["ue8m0"] else t


def _source_rows(s, at, live):
    return s["index"].long()[torch.where(live, at, 0)] if s["case"]["gather"] else at


def _plain(s):
    c, kind = s["case"], s["case"]["kind"]
    if kind == "order":
        b, n, sr, rs = _order(s["topk"], s["offset"], c, s["slots"])
        return b.int(), n.int(), sr.int(), rs.int()
    if kind == "reduce":
        used = (s["row_slot"] >= 0).unsqueeze(2)
        z = s["z"][s["row_slot"].clamp_min(0).long()].float().masked_fill_(~used, 0.0)
        return (z * s["weights"].unsqueeze(2)).sum(1).to(torch.bfloat16)
    if kind == "reduce_bwd":
        used = s["row_slot"] >= 0
        place = torch.where(used, s["row_slot"].long(), s["slots"]).reshape(-1)
        dy = s["dy"].float()
        dz = torch.zeros((s["slots"] + 1, c["H"]), dtype=torch.bfloat16, device="cuda")  # the last: entries without a slot
        dz[place] = (dy.unsqueeze(1) * s["weights"].unsqueeze(2)).to(torch.bfloat16).reshape(-1, c["H"])
        z = s["z"][s["row_slot"].clamp_min(0).long()].float().masked_fill_(~used.unsqueeze(2), 0.0)
        return dz[:-1], (z * dy.unsqueeze(1)).sum(2)
    if kind.startswith("swiglu"):
        live = _live_rows(s)
        h = s["h"].float()
        gate, up = h[:, :c["I"]], h[:, c["I"]:]
        sig = 1.0 / (1.0 + torch.exp(-gate))
        if kind == "swiglu_bwd":
            da = s["da"].float()
            dgate = da * up * sig * (1.0 + gate * (1.0 - sig))
            return torch.cat([dgate, da * gate * sig], 1).masked_fill_(~live, 0.0).to(torch.bfloat16)
        a = (gate * sig * up).masked_fill_(~live, 0.0)
        if not c["fp8"]:
            return a.to(torch.bfloat16)
        v = a.view(a.shape[0], -1, 128)
        amax = v.abs().amax(2).clamp_min(1e-4)
        code = (v * (448.0 / amax).unsqueeze(2)).view(a.shape).to(FP8)
        return code, (amax / 448.0).masked_fill_(~live, 0.0)
    at, live = _padded(s)
    if kind == "dgrad":
        return _put(at, torch.bmm(_take(s["dy"], at, live), s["w"].float()), s["total"], torch.bfloat16)
    x = _take(s["x"], _source_rows(s, at, live), live)
    if kind == "wgrad":
        return torch.bmm(_take(s["dy"], at, live).transpose(1, 2).contiguous(), x)
    w = s["w"].float()
    if kind == "fp8":
        xs = _take(_scales(s, s["x_scales"]), _source_rows(s, at, live), live)
        x = (x.view(*x.shape[:2], -1, 128) * xs.unsqueeze(3)).view(x.shape)
        ws = _scales(s, s["w_scales"]).repeat_interleave(128, 1)[:, :c["N"]]
        w = (w.view(c["G"], c["N"], -1, 128) * ws.unsqueeze(3)).view(w.shape)
    return _put(at, torch.bmm(x, w.transpose(1, 2).contiguous()), s["total"], torch.bfloat16)


# ------------------------------------------------------------------ the package's calls
def _own(s):
    import combine_get_dispatch_histogram_amd as miep
    c, kind = s["case"], s["case"]["kind"]
    if kind in ("order", "reduce", "reduce_bwd"):
        order = miep.ExpertOrder(group_begin=s["begin"], group_rows=s["count"], slot_row=s["slot_row"], row_slot=s["row_slot"],
                                 recv_rank_offset=s["offset"], workspace=s["workspace"])
        if kind == "order":
            miep.expert_order_into(s["topk"], order, expert_alignment=c["align"])
            return s["begin"], s["count"], s["slot_row"], s["row_slot"]
        if kind == "reduce":
            miep.expert_reduce_into(s["z"], order, s["y"], topk_weights=s["weights"])
            return s["y"]
        miep.expert_reduce_backward_into(s["dy"], s["z"], order, s["dz"], topk_weights=s["weights"], d_topk_weights=s["dw"])
        return s["dz"], s["dw"]
    groups = miep.RowGroups(rows=s["count"], begin=s["begin"])
    if kind == "swiglu_bwd":
        miep.swiglu_backward_into(s["da"], s["h"], groups, s["dh"])
        return s["dh"]
    if kind == "swiglu":
        if c["fp8"]:
            miep.swiglu_fp8_into(s["h"], groups, s["a"], s["scales"])
            return s["a"], s["scales"]
        miep.swiglu_into(s["h"], groups, s["a"])
        return s["a"]
    if kind == "dgrad":
        miep.grouped_gemm_dgrad_into(s["dy"], s["w"], groups, s["dx"], expected_rows=s["expected"])
        return s["dx"]
    if kind == "wgrad":
        miep.grouped_gemm_wgrad_into(s["dy"], s["x"], groups, s["dweight"], row_index=s.get("index"))
        return s["dweight"]
    if kind == "fp8":
        miep.grouped_gemm_fp8_into(s["x"], s["x_scales"], s["w"], s["w_scales"], groups, s["y"], row_index=s.get("index"),
                                   expected_rows=s["expected"])
        return s["y"]
    miep.grouped_gemm_into(s["x"], s["w"], groups, s["y"], row_index=s.get("index"), expected_rows=s["expected"])
    return s["y"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def work(case):
    c, kind = case, case["kind"]
    if kind in ("order", "reduce", "reduce_bwd"):
        wide = c["E"] * 8 if c["routing"] == "masked" else c["E"]
        entries = c["N"] * c["K"] * c["E"] / wide                              # slots
        share = c["E"] / c["R"] / wide                                         # of the experts, on one rank
        rows = c["N"] * c["R"] * (1 - (1 - share) ** c["K"])                   # rows that are received, about
        if kind == "order":
            return dict(bytes=rows * c["K"] * 12 + entries * 4 + c["E"] * 8, flops=0)
        meta = rows * c["K"] * 8
        if kind == "reduce":
            return dict(bytes=meta + 2 * c["H"] * (entries + rows), flops=2 * entries * c["H"])
        return dict(bytes=meta * 1.5 + 2 * c["H"] * (2 * entries + rows), flops=3 * entries * c["H"])
    G, rows = c["G"], c["rows"]
    if kind.startswith("swiglu"):
        out = 6 * c["I"] if kind == "swiglu_bwd" else (c["I"] + c["I"] // 32 if c["fp8"] else 2 * c["I"])
        return dict(bytes=rows * (4 * c["I"] + out), flops=8 * rows * c["I"])
    N, K = c["N"], c["K"]
    src = rows // 2 if c["gather"] else rows
    flops = 2 * rows * N * K
    live = min(G, rows) if c["dist"] == "even" else max(1, G - 1)
    if kind == "fp8":
        return dict(bytes=live * N * K + src * K + 2 * rows * N, flops=flops)
    if kind == "wgrad":
        return dict(bytes=4 * G * N * K + 2 * (src * K + rows * N), flops=flops)
    return dict(bytes=2 * (live * N * K + src * K + rows * N), flops=flops)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s, c, kind = prepare(case, seed), case, case["kind"]
    if kind == "order":
        return None
    if kind in ("reduce", "reduce_bwd"):
        slot, w = s["row_slot"].long(), s["weights"].double()
        if kind == "reduce":
            out = torch.zeros((slot.shape[0], c["H"]), dtype=torch.float64, device="cuda")
            for k in range(c["K"]):
                live = slot[:, k] >= 0
                out[live] += w[live, k, None] * s["z"][slot[live, k]].double()
            return out
        dz = torch.zeros((s["slots"], c["H"]), dtype=torch.float64, device="cuda")
        dw = torch.zeros_like(w)
        for k in range(c["K"]):
            live = slot[:, k] >= 0
            dy = s["dy"][live].double()
            dz[slot[live, k]] = w[live, k, None] * dy
            dw[live, k] = (dy * s["z"][slot[live, k]].double()).sum(1)
        return dz, dw
    out, sc = None, None
    for g, (b, n) in enumerate(zip(s["begin"].tolist(), s["count"].tolist())):
        at = torch.arange(b, b + n, device="cuda")
        src = s["index"][at].long() if c.get("gather") else at
        if kind.startswith("swiglu"):
            I = c["I"]
            gate, up = s["h"][at, :I].double(), s["h"][at, I:].double()
            sig = torch.sigmoid(gate)
            if kind == "swiglu_bwd":
                da = s["da"][at].double()
                v = torch.cat([da * up * (sig + gate * sig * (1 - sig)), da * gate * sig], 1)
            else:
                v = gate * sig * up
                if c["fp8"]:
                    top = v.view(n, -1, 128).abs().amax(2).clamp_min(1e-4)
                    v = (v.view(n, -1, 128) / top.unsqueeze(2) * 448).view(n, I)
                    sc = torch.zeros((s["total"], I // 128), dtype=torch.float64, device="cuda") if sc is None else sc
                    sc[at] = top / 448
        elif kind == "dgrad":
            v = s["dy"][at].double() @ s["w"][g].double()
        elif kind == "wgrad":
            v = s["dy"][at].double().t().contiguous() @ s["x"][src].double()
            out = torch.zeros((c["G"], c["N"], c["K"]), dtype=torch.float64, device="cuda") if out is None else out
            out[g] = v
            continue
        elif kind == "gemm":
            v = s["x"][src].double() @ s["w"][g].double().t().contiguous()
        else:
            e2 = (lambda t: torch.exp2(t.double() - 127)) if c["ue8m0"] else (lambda t: t.double())
            x = s["x"][src].double() * e2(s["x_scales"][src]).repeat_interleave(128, 1)
            w = s["w"][g].double() * e2(s["w_scales"][g]).repeat_interleave(128, 0)[:c["N"]].repeat_interleave(128, 1)
            v = x @ w.t().contiguous()
        out = torch.zeros((s["total"], v.shape[1]), dtype=torch.float64, device="cuda") if out is None else out
        out[at] = v
    return out if sc is None else (out, sc)
