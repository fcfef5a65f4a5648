"""Cases of the mixture-of-experts operators around the grouped products, and of
the forward of few rows from 4-bit weights: what each call is given, its plain
form in elementary fp32 torch operations, and its exact result.

Operators (names as in the package):
  gate      lp_moe_gate: softmax over a token's expert logits, the k largest
            (ties to the lowest index, -inf never chosen), their weights;
            train: lp_moe_gate_bwd too
  dispatch  lp_moe_sort (the (token, slot) pairs stably sorted by expert;
            experts outside 0 .. E-1 are nobody's), then the rows in that
            order: lp_moe_gather, or lp_moe_gather_quant straight into the
            two E4M3 copies that grouped products take; train: the gradient
            of the tokens from that of the rows too
  combine   lp_moe_combine: every token's rows summed by their weights;
            train: lp_moe_combine_bwd too, fp8: its gradient of the rows in
            the two E4M3 copies
  w4        lp_linear_fwd_w4, lp_grouped_fwd_w4: y = x @ W^T, x bf16, W E2M1
            with an E8M0 scale per 32 (mxfp4), or an E4M3 scale per 16 and one
            fp32 scale (nvfp4); an element is bf16(fp32(code * scale))
"""
import math

import torch

own = False

RUN = 128
E4M3_MAX = 448.0
FLOOR = 2.0 ** -64
F8 = torch.float8_e4m3fn
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
BF = torch.bfloat16


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token's choice of 8 among 64 experts: a decoding step, latency
        {"name": "gate_token", "op": "gate", "T": 1, "E": 64, "k": 8, "type": "f32", "renorm": True, "mask": 0.0, "train": False},
        # a training batch over 256 experts, the softmax's own weights, with its gradient
        {"name": "gate_train", "op": "gate", "T": 32768, "E": 256, "k": 8, "type": "bf16", "renorm": False, "mask": 0.0,
         "train": True},
        # a decoding batch of 12 tokens to 8 of 64 experts: 96 rows
        {"name": "dispatch_decode", "op": "dispatch", "T": 12, "k": 8, "E": 64, "H": 7168, "route": "zipf", "drop": 0.0,
         "fp8": False, "train": False},
        # a short ragged batch, some experts on another machine, with its gradient
        {"name": "dispatch_ragged", "op": "dispatch", "T": 1000, "k": 6, "E": 40, "H": 1040, "route": "dirichlet", "drop": 0.2,
         "fp8": False, "train": True},
        # a training batch to 8 of 64 experts in FP8: 32768 rows
        {"name": "dispatch_fp8", "op": "dispatch", "T": 4096, "k": 8, "E": 64, "H": 7168, "route": "zipf", "drop": 0.0,
         "fp8": True, "train": False},
        # the decoding batch's way back
        {"name": "combine_decode", "op": "combine", "T": 12, "k": 8, "E": 64, "H": 7168, "route": "zipf", "drop": 0.0,
         "fp8": False, "train": False},
        # a training batch to 2 of 8 experts: 16384 rows there and back
        {"name": "combine_train", "op": "combine", "T": 8192, "k": 2, "E": 8, "H": 4096, "route": "dirichlet", "drop": 0.0,
         "fp8": False, "train": True},
        # the 64 experts' way back, its gradient in FP8
        {"name": "combine_fp8", "op": "combine", "T": 4096, "k": 8, "E": 64, "H": 7168, "route": "zipf", "drop": 0.0,
         "fp8": True, "train": True},
        # one token through a 4096 x 4096 projection: a decoding step, latency
        {"name": "w4_token", "op": "w4", "M": 1, "N": 4096, "K": 4096, "fmt": "mxfp4"},
        # a small decoding batch through the 8192 x 2048 projection
        {"name": "w4_batch", "op": "w4", "M": 24, "N": 8192, "K": 2048, "fmt": "nvfp4"},
        # a prompt through a layer of odd sizes
        {"name": "w4_prompt", "op": "w4", "M": 1000, "N": 4112, "K": 4128, "fmt": "mxfp4"},
        # decoding through 64 experts: a few rows each, most weights read once
        {"name": "w4_experts", "op": "w4", "M": 96, "N": 2048, "K": 7168, "G": 64, "fmt": "nvfp4", "route": "zipf"},
    ]


def _log(rng, lo, hi, mul=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v) // mul * mul))


def draw(rng):
    op = rng.choice(["gate", "dispatch", "combine", "w4", "w4"])
    if op == "gate":
        E = _log(rng, 2, 1024)
        return {"op": op, "T": _log(rng, 1, min(32768, (1 << 23) // E)), "E": E, "k": rng.randint(1, min(16, E)),
                "type": rng.choice(["f32", "bf16"]), "renorm": rng.random() < 0.5, "mask": rng.choice([0.0, 0.0, 0.3, 0.9]),
                "train": rng.random() < 0.5}
    if op == "w4":
        while True:
            c = {"op": op, "M": _log(rng, 1, 2048), "N": _log(rng, 128, 8192, 16), "K": _log(rng, 128, 8192, 32),
                 "fmt": rng.choice(["mxfp4", "nvfp4"])}
            if rng.random() < 0.5:
                c["G"], c["route"] = _log(rng, 1, 64), rng.choice(["zipf", "dirichlet", "even"])
            if c["M"] * c["N"] * c["K"] <= 1 << 34 and c.get("G", 1) * c["N"] * c["K"] <= 1 << 29:
                return c
    while True:
        c = {"op": op, "T": _log(rng, 1, 16384), "k": rng.randint(1, 8), "E": _log(rng, 1, 256), "H": _log(rng, 16, 8192, 16),
             "route": rng.choice(["zipf", "dirichlet", "even"]), "drop": rng.choice([0.0, 0.0, 0.1, 0.5]),
             "fp8": rng.random() < 0.4, "train": rng.random() < 0.5}
        if c["k"] <= c["E"] and c["T"] * c["k"] * c["H"] <= 1 << 26:
            return c


def _popularity(route, E, gen):
    """How much each expert is asked for."""
    if route == "zipf":
        return torch.arange(1, E + 1, dtype=torch.float64).pow(-1.1)[torch.randperm(E, generator=gen)]
    if route == "dirichlet":
        return -torch.rand(E, generator=gen, dtype=torch.float64).clamp_min(1e-12).log()
    return torch.ones(E, dtype=torch.float64)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    return {"gate": _prepare_gate, "w4": _prepare_w4}.get(case["op"], _prepare_rows)(case, seed, gen, randn)


def _prepare_gate(case, seed, gen, randn):
    T, E, k = case["T"], case["E"], case["k"]
    logits = randn(T, E) * 1.5 + randn(1, E)                  # some experts are liked by most tokens
    if case["mask"]:
        away = torch.rand(T, E, generator=gen, device="cuda") < case["mask"]
        away[0] = True                                        # a padding token: nobody's
        logits.masked_fill_(away, -math.inf)
    logits = logits.to(BF) if case["type"] == "bf16" else logits
    return {"op": "gate", "logits": logits, "k": k, "renorm": case["renorm"], "grad": randn(T, k) if case["train"] else None}


def _prepare_rows(case, seed, gen, randn):
    T, k, E, H = case["T"], case["k"], case["E"], case["H"]
    host = torch.Generator().manual_seed(seed)
    # k different experts for every token, the popular ones more often (the largest of logs plus exponential noise)
    score = _popularity(case["route"], E, host).log().float().cuda() - torch.empty(T, E, device="cuda").exponential_(generator=gen).log()
    experts = score.topk(k, dim=1).indices.to(torch.int32)
    experts[torch.rand(T, k, generator=gen, device="cuda") < case["drop"]] = -1
    s = {"op": case["op"], "fp8": case["fp8"], "train": case["train"], "E": E, "k": k, "experts": experts}
    act = (1 + 9 * (torch.rand(H, generator=gen, device="cuda") < 0.01)).to(torch.float32)    # a few outlier channels
    M = T * k
    if case["op"] == "dispatch":
        s["x"] = (randn(T, H) * act).to(BF)
        if case["train"]:
            s["grad_rows"] = (randn(M, H) * 1e-3).to(BF)
    else:
        s["offsets"], s["rows"], s["pairs"] = _plain_sort(experts, E)
        s["y"] = (randn(M, H) * act).to(BF)
        s["weights"] = torch.softmax(randn(T, k), 1)
        if case["train"]:
            s["grad"] = (randn(T, H) * 1e-3 * randn(T, 1).mul_(0.5).exp_()).to(BF)
    # buffers that a training loop keeps: rows past the last expert's stay as they are
    if case["fp8"]:
        s["cols"] = (torch.zeros(1, M, H, dtype=torch.uint8, device="cuda"), torch.zeros(1, -(-H // RUN), M, device="cuda"))
        s["tokens"] = (torch.zeros(1, M, H, dtype=torch.uint8, device="cuda"), torch.zeros(1, M // RUN + E, H, device="cuda"))
    else:
        s["out"] = torch.zeros(M, H, dtype=BF, device="cuda")
    return s


def _ends(case):
    """Cumulative ends of the experts' rows: loads by the case's routing, the same for every seed."""
    G, M = case.get("G", 1), case["M"]
    g = torch.Generator().manual_seed(1000 + G + M)
    pick = torch.multinomial(_popularity(case.get("route"), G, g), M, replacement=True, generator=g)
    return torch.bincount(pick, minlength=G).cumsum(0).tolist()


def _prepare_w4(case, seed, gen, randn):
    M, N, K, G, fmt = case["M"], case["N"], case["K"], case.get("G", 1), case["fmt"]
    block = 32 if fmt == "mxfp4" else 16
    codes = torch.empty(G, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(G, N, K // block, dtype=torch.uint8, device="cuda")
    ts = torch.full((1,), 0.1 / (6 * 448), device="cuda")    # the largest weight over the largest value
    for g in range(G):
        v = randn(N, K // block, block).mul_(0.02)
        a = v.abs().amax(-1)
        if fmt == "mxfp4":
            e = torch.frexp(a)[1] - 3                         # the largest falls into [4, 8)
            scales[g] = (e + 127).to(torch.uint8)
            step = torch.exp2(e.float())
        else:
            f8 = (a / 6 / ts).clamp(2.0 ** -9, E4M3_MAX).to(F8)
            scales[g] = f8.view(torch.uint8)
            step = f8.float() * ts
        v = v / step[..., None]
        c = torch.bucketize(v.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")).to(torch.uint8)
        c = (c | ((v < 0).to(torch.uint8) << 3)).view(N, K)
        codes[g] = c[:, 0::2] | (c[:, 1::2] << 4)
    x = (randn(M, K) * (1 + 9 * (torch.rand(K, generator=gen, device="cuda") < 0.01))).to(BF)
    ends = _ends(case)
    return {"op": "w4", "fmt": fmt, "grouped": "G" in case, "x": x, "codes": codes, "scales": scales,
            "ts": ts if fmt == "nvfp4" else None, "ends": ends, "offsets": torch.tensor(ends, dtype=torch.int32, device="cuda")}


# ---------------------------------------------------------------- plain forms

def _plain_gate(s):
    logits, k = s["logits"].float(), s["k"]
    top, at = torch.sort(logits, dim=1, descending=True, stable=True)
    top, at = top[:, :k], at[:, :k]
    none = top == -math.inf
    peak = torch.where(none[:, :1], 0.0, top[:, :1])
    e = torch.exp(logits - peak)
    total = e.sum(1, keepdim=True)
    chosen = torch.exp(top - peak)                            # 0 where none
    w = chosen / (chosen.sum(1, keepdim=True) if s["renorm"] else total).clamp_min(1e-38)
    out = {"weights": w, "experts": torch.where(none, -1, at).to(torch.int32)}
    if s["grad"] is not None:
        dw = torch.where(none, 0.0, s["grad"])
        inner = (w * dw).sum(1, keepdim=True)
        p = torch.zeros_like(logits) if s["renorm"] else e / total.clamp_min(1e-38) * -inner
        p.scatter_add_(1, at, w * (dw - inner) if s["renorm"] else w * dw)
        out["grad"] = p.to(s["logits"].dtype)
    return out


def _plain_sort(experts, E):
    """offsets, the row of every pair (-1: nobody's), the pair of every row (those past the last expert's in any order)."""
    flat = experts.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < E), flat, E)
    _, pairs = torch.sort(flat, stable=True)
    offsets = (flat[None] == torch.arange(E, device=flat.device)[:, None]).sum(1).cumsum(0)
    rows = torch.empty_like(flat)
    rows[pairs] = torch.arange(flat.numel(), device=flat.device)
    rows = torch.where(flat < E, rows, -1)
    return offsets.to(torch.int32), rows.view(experts.shape).to(torch.int32), pairs.to(torch.int32)


def _run_of_row(offsets, M):
    """The run index of every row: group g's runs start at first_row // 128 + g."""
    row = torch.arange(M, dtype=torch.int32, device=offsets.device)
    g = torch.searchsorted(offsets, row, right=True)
    first = torch.cat([offsets.new_zeros(1), offsets])[g]
    return (first // RUN + g + (row - first) // RUN).long()


def _scale(amax):
    return torch.div(amax.clamp_min(FLOOR), amax.new_full((), E4M3_MAX))


def _code(v, s):
    return torch.div(v, s).clamp_(-E4M3_MAX, E4M3_MAX).to(F8)


def _plain_quant(s, v, live, offsets):
    """Both E4M3 copies of the rows v [M, H] that `live` marks, into the state's buffers."""
    M, H = v.shape
    nb = -(-H // RUN)
    pad = torch.nn.functional.pad(v, (0, nb * RUN - H)).view(M, nb, RUN)
    sc = _scale(pad.abs().amax(-1, keepdim=True))
    keep = live[:, None]
    s["cols"][0].view(F8)[0] = torch.where(keep, _code(pad, sc).view(M, -1)[:, :H].float(), 0.0).to(F8)
    s["cols"][1][0] = torch.where(keep, sc.view(M, nb), 0.0).t()
    run = _run_of_row(offsets, M).clamp_max(s["tokens"][1].shape[1] - 1)
    amax = v.new_full((s["tokens"][1].shape[1], H), -1.0).index_reduce_(0, run, torch.where(keep, v.abs(), -1.0), "amax")
    sc = torch.where(amax < 0, 0.0, _scale(amax))
    s["tokens"][0].view(F8)[0] = torch.where(keep, _code(v, sc[run]).float(), 0.0).to(F8)
    s["tokens"][1][0] = sc


def _fp8_outputs(s):
    return {"cols": s["cols"][0].view(F8), "cols_scales": s["cols"][1], "tokens": s["tokens"][0].view(F8),
            "tokens_scales": s["tokens"][1]}


def _plain_dispatch(s):
    offsets, rows, pairs = _plain_sort(s["experts"], s["E"])
    live = torch.arange(pairs.numel(), device=pairs.device) < offsets[-1]
    v = s["x"][(pairs // s["k"]).long()]
    out = {"offsets": offsets, "rows": rows}
    if s["fp8"]:
        _plain_quant(s, v.float(), live, offsets)
        out.update(_fp8_outputs(s))
    else:
        s["out"].copy_(torch.where(live[:, None], v, 0))
        out["x"] = s["out"]
    if s["train"]:
        out["grad"] = _plain_sum(s["grad_rows"], rows, None).to(BF)
    return out


def _plain_sum(y, rows, weights):
    total = 0
    for j in range(rows.shape[1]):
        part = torch.where(rows[:, j, None] >= 0, y[rows[:, j].clamp_min(0).long()].float(), 0.0)
        total = total + (part if weights is None else part * weights[:, j, None])
    return total


def _plain_combine(s):
    rows, w, y, k = s["rows"], s["weights"], s["y"], s["k"]
    out = {"y": _plain_sum(y, rows, w).to(BF)}
    if s["train"]:
        pairs = s["pairs"].long()
        live = torch.arange(pairs.numel(), device=pairs.device) < s["offsets"][-1]
        token = pairs // k
        g = s["grad"][token].float()
        dot = (g * torch.where(live[:, None], y.float(), 0.0)).sum(1)
        out["grad_weights"] = torch.empty_like(w).view(-1).index_copy_(0, pairs, dot).view_as(w)
        v = (g * w.reshape(-1)[pairs][:, None]).to(BF)
        if s["fp8"]:
            _plain_quant(s, v.float(), live, s["offsets"])
            out.update(_fp8_outputs(s))
        else:
            s["out"].copy_(torch.where(live[:, None], v, 0))
            out["grad_y"] = s["out"]
    return out


def _decode4(fmt, codes, scales, ts):
    """[N, K / 2] bytes -> fp32 [N, K], every element rounded to bf16."""
    lut = torch.tensor(E2M1 + [-v for v in E2M1], device=codes.device)
    v = lut[torch.stack([codes & 15, codes >> 4], -1).long()].view(codes.shape[0], -1)
    s = torch.exp2(scales.float() - 127) if fmt == "mxfp4" else scales.view(F8).float() * ts
    return (v * s.repeat_interleave(32 if fmt == "mxfp4" else 16, 1)).to(BF).float()


def _plain_w4(s):
    x = s["x"].float()
    y = torch.empty(x.shape[0], s["codes"].shape[1], dtype=BF, device=x.device)
    for g, (a, b) in enumerate(zip([0] + s["ends"], s["ends"])):
        if b > a:
            y[a:b] = x[a:b] @ _decode4(s["fmt"], s["codes"][g], s["scales"][g], s["ts"]).t()
    return {"y": y}


# ---------------------------------------------------------------- the framework's calls

def _own_gate(s):
    import fp8_gemm_backward_amd as lp
    w, e = lp.lp_moe_gate(s["logits"], s["k"], renorm=s["renorm"])
    out = {"weights": w, "experts": e}
    if s["grad"] is not None:
        out["grad"] = lp.lp_moe_gate_bwd(s["grad"], s["logits"], w, e, renorm=s["renorm"])
    return out


def _own_quant(lp, s, x, pairs, offsets, weights=None):
    cols = lp.QTensor("fp8_r128", *s["cols"], axis=-1)
    tokens = lp.QTensor("fp8_r128", *s["tokens"], axis=-2)
    lp.lp_moe_gather_quant(x, pairs, offsets, s["k"], weights=weights, out=(cols, tokens))
    return _fp8_outputs(s)


def _own_dispatch(s):
    import fp8_gemm_backward_amd as lp
    offsets, rows, pairs = lp.lp_moe_sort(s["experts"], s["E"])
    out = {"offsets": offsets, "rows": rows}
    if s["fp8"]:
        out.update(_own_quant(lp, s, s["x"], pairs, offsets))
    else:
        out["x"] = lp.lp_moe_gather(s["x"], rows, out=s["out"])
    if s["train"]:
        out["grad"] = lp.lp_moe_combine(s["grad_rows"], rows)
    return out


def _own_combine(s):
    import fp8_gemm_backward_amd as lp
    out = {"y": lp.lp_moe_combine(s["y"], s["rows"], s["weights"])}
    if s["train"] and s["fp8"]:
        out["grad_weights"] = lp.lp_moe_combine_bwd(s["grad"], s["y"], s["rows"], s["weights"], need_dy=False)[1]
        out.update(_own_quant(lp, s, s["grad"], s["pairs"], s["offsets"], s["weights"]))
    elif s["train"]:
        out["grad_y"], out["grad_weights"] = lp.lp_moe_combine_bwd(s["grad"], s["y"], s["rows"], s["weights"], grad_y=s["out"])
    return out


def _own_w4(s):
    import fp8_gemm_backward_amd as lp
    w = lp.QTensor(s["fmt"], s["codes"], s["scales"], s["ts"])
    return {"y": lp.lp_grouped_fwd_w4(s["x"], w, s["offsets"]) if s["grouped"] else lp.lp_linear_fwd_w4(s["x"], w)}


def run(state):
    plain = {"gate": _plain_gate, "dispatch": _plain_dispatch, "combine": _plain_combine, "w4": _plain_w4}
    mine = {"gate": _own_gate, "dispatch": _own_dispatch, "combine": _own_combine, "w4": _own_w4}
    return (mine if own else plain)[state["op"]](state)


# ---------------------------------------------------------------- work and exact results

def work(case):
    op = case["op"]
    if op == "gate":
        T, E, k, size = case["T"], case["E"], case["k"], 2 if case["type"] == "bf16" else 4
        fwd = T * E * size + 8 * T * k
        return {"bytes": fwd + (T * E * size + 4 * T * k if case["train"] else 0), "flops": 4 * T * E * (2 if case["train"] else 1)}
    if op == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        ends = _ends(case)
        used = sum(b > a for a, b in zip([0] + ends, ends))      # an expert without a row is not read
        return {"bytes": used * (N * K // 2 + N * K // (32 if case["fmt"] == "mxfp4" else 16)) + 2 * M * K + 2 * M * N,
                "flops": 2 * M * N * K}
    T, H, M = case["T"], case["H"], case["T"] * case["k"]
    live = round(M * (1 - case["drop"]))
    rows, tokens = 2 * live * H, 2 * T * H
    both = 2 * live * H + 8 * live * H // RUN                    # two copies of a byte an element, and their scales
    if op == "dispatch":
        return {"bytes": 12 * M + tokens + (both if case["fp8"] else rows) + (rows + tokens if case["train"] else 0),
                "flops": live * H * ((6 if case["fp8"] else 0) + (1 if case["train"] else 0))}
    b, f = 8 * M + rows + tokens, 2 * live * H
    if case["train"]:
        b, f = b + tokens + 4 * M + (both if case["fp8"] else rows), f + live * H * (9 if case["fp8"] else 3)
    return {"bytes": b, "flops": f}


def _exact_gate(s):
    l = s["logits"].double()
    T, E = l.shape
    left, e, v = l.clone(), [], []
    for _ in range(s["k"]):                                      # the largest, then the largest of the rest
        m = left.amax(1)
        at = torch.where(left == m[:, None], torch.arange(E, device=l.device), E).amin(1)
        e.append(torch.where(m == -math.inf, -1, at))
        v.append(m)
        left.scatter_(1, at[:, None], -math.inf)
    e, v = torch.stack(e, 1), torch.stack(v, 1)
    base = torch.where(e[:, :1] < 0, 0.0, l.amax(1, keepdim=True))
    num = torch.exp(v - base)
    whole = torch.exp(l - base)
    den = num.sum(1, keepdim=True) if s["renorm"] else whole.sum(1, keepdim=True)
    w = torch.where(e < 0, 0.0, num / den)
    out = {"weights": w, "experts": e.to(torch.int32)}
    if s["grad"] is not None:
        # d w_j / d l_i = w_j ([i = e_j] - q_i), q: the softmax whose denominator w_j has
        dw = s["grad"].double()
        hit = torch.zeros(T, E, dtype=torch.float64, device=l.device)
        q = torch.zeros_like(hit)
        for j in range(s["k"]):
            ok = (e[:, j] >= 0).double()[:, None]
            one = torch.zeros_like(hit).scatter_(1, e[:, j, None].clamp_min(0), ok)
            hit += one * (w[:, j] * dw[:, j])[:, None]
            q += one * w[:, j, None]
        if not s["renorm"]:
            q = torch.where(den > 0, whole / den, 0.0)
        out["grad"] = hit - q * hit.sum(1, keepdim=True)
    return out


def _exact_order(experts, E):
    """By counting, expert by expert, on the host."""
    e = experts.reshape(-1).cpu()
    rows, at, ends = torch.full_like(e, -1), 0, []
    for g in range(E):
        mine = (e == g).nonzero()[:, 0]
        rows[mine] = torch.arange(at, at + mine.numel(), dtype=rows.dtype)
        at += mine.numel()
        ends.append(at)
    return ends, rows.view(experts.shape).cuda()


def _nearest_e4m3(t):
    """E4M3 rounding of 64-bit values from its definition: 3 mantissa bits, exponents from -6, ties to even, at most 448."""
    _, e = torch.frexp(t)
    unit = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return (torch.round(t / unit) * unit).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_run(v, dim):
    """Codes and scale of one run along dim: the stated fp32 roundings, everything else in 64 bits."""
    sc = (v.abs().amax(dim, keepdim=True).clamp_min(FLOOR) / E4M3_MAX).float().double()
    return _nearest_e4m3((v / sc).float().double()), sc


def _exact_quant(s, v, ends):
    """v in 64 bits [M, H]: both copies, run by run; what no expert has is 0."""
    M, H = v.shape
    cols, cs = torch.zeros_like(v), torch.zeros(1, -(-H // RUN), M, dtype=v.dtype, device=v.device)
    for b in range(0, H, RUN):
        q, sc = _exact_run(v[:ends[-1], b:b + RUN], 1) if ends[-1] else (0, 0)
        if ends[-1]:
            cols[:ends[-1], b:b + RUN], cs[0, b // RUN, :ends[-1]] = q, sc[:, 0]
    toks, tsc = torch.zeros_like(v), torch.zeros(1, M // RUN + s["E"], H, dtype=v.dtype, device=v.device)
    for g, (a, z) in enumerate(zip([0] + ends, ends)):
        for i in range(a, z, RUN):
            q, sc = _exact_run(v[i:min(i + RUN, z)], 0)
            toks[i:min(i + RUN, z)], tsc[0, a // RUN + g + (i - a) // RUN] = q, sc[0]
    cols[ends[-1]:] = 0
    return {"cols": cols[None], "cols_scales": cs, "tokens": toks[None], "tokens_scales": tsc}


def _exact_rows(s):
    ends, rows = _exact_order(s["experts"], s["E"])
    T, k = rows.shape
    dispatch = s["op"] == "dispatch"
    src = s["x"].double() if dispatch else s["grad"].double() if s["train"] else None
    M = T * k
    out = {"offsets": torch.tensor(ends, dtype=torch.int32, device="cuda"), "rows": rows} if dispatch else {}
    if src is not None:
        v = torch.zeros(M, src.shape[1], dtype=torch.float64, device="cuda")
        for j in range(k):
            ok = rows[:, j] >= 0
            part = src[ok]
            if not dispatch:
                part = part * s["weights"][ok, j, None].double()
                if s["fp8"]:
                    part = part.float().to(BF).double()          # quantized from bf16
            v[rows[ok, j].long()] = part
        if s["fp8"]:
            out.update(_exact_quant(s, v, ends))
        else:
            out["x" if dispatch else "grad_y"] = v
    if dispatch and not s["train"]:
        return out
    y = (s["grad_rows"] if dispatch else s["y"]).double()
    total = torch.zeros(T, y.shape[1], dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        ok = rows[:, j] >= 0
        mine = y[rows[ok, j].long()]
        total[ok] += mine if dispatch else mine * s["weights"][ok, j, None].double()
        if not dispatch and s["train"]:
            dw[ok, j] = (mine * src[ok]).sum(1)
    out["grad" if dispatch else "y"] = total
    if not dispatch and s["train"]:
        out["grad_weights"] = dw
    return out


def _exact_w4(s):
    x = s["x"].double()
    M, (G, N, half) = x.shape[0], s["codes"].shape
    y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for g, (a, b) in enumerate(zip([0] + s["ends"], s["ends"])):
        if b <= a:
            continue
        w = torch.empty(N, 2 * half, dtype=torch.float64, device="cuda")
        for odd in (0, 1):
            c = (s["codes"][g] >> (4 * odd)) & 15
            man, ex, sign = (c & 1).double(), ((c >> 1) & 3).double(), 1 - 2 * (c >> 3).double()
            w[:, odd::2] = sign * torch.where(ex == 0, man * 0.5, (1 + man / 2) * torch.exp2(ex - 1))
        if s["fmt"] == "mxfp4":
            sc, block = torch.exp2(s["scales"][g].double() - 127), 32
        else:
            sc, block = (s["scales"][g].view(F8).double() * s["ts"].double()).float().double(), 16
        w = (w.view(N, -1, block) * sc[..., None]).float().to(BF).double().view(N, -1)      # an element's stated roundings
        y[a:b] = x[a:b] @ w.t()
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    return {"gate": _exact_gate, "w4": _exact_w4}.get(s["op"], _exact_rows)(s)
