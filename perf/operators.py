"""Cases of the block-scaled FP8 training operators: what each call is given,
its plain form in elementary fp32 torch operations, and its exact result.

Operators (names as in the package):
  linear_fwd    y = x @ W^T: bf16 x quantized to E4M3 with an fp32 scale per
                run of 128 along K, W E4M3 with an fp32 scale per 128 x 128 block
  linear_bwd    bf16 gradient quantized along N and along the tokens;
                grad_X = grad @ W, grad_W = grad^T @ x, x kept quantized along
                the tokens
  grouped_fwd,  the same per expert, rows grouped by int32 cumulative ends;
  grouped_bwd   runs along the tokens restart at each group's first row
  adamw         one AdamW step over many tensors, moments in fp32 or in E4M3
                with an fp32 scale per run of 128

Quantization of a run (or block) with largest magnitude a:
s = fp32(max(a, 2^-64) / 448), code = E4M3(fp32(v / s)).
"""
import math

import torch

own = False

RUN = 128
E4M3_MAX = 448.0
FLOOR = 2.0 ** -64
F8 = torch.float8_e4m3fn

BETA1, BETA2, EPS, LR, DECAY, STEP = 0.9, 0.95, 1e-8, 3e-4, 0.1, 7


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token through a 4096 x 4096 projection: a decoding step, latency
        {"name": "fwd_token", "op": "linear_fwd", "M": 1, "N": 4096, "K": 4096},
        # a small decoding batch through the 8192 x 2048 projection
        {"name": "fwd_batch", "op": "linear_fwd", "M": 24, "N": 8192, "K": 2048},
        # a training batch through the same layer
        {"name": "fwd_train", "op": "linear_fwd", "M": 4096, "N": 8192, "K": 2048},
        # a short ragged batch, no size a multiple of 128
        {"name": "bwd_ragged", "op": "linear_bwd", "M": 1000, "N": 2064, "K": 1040},
        # the square 4096 layer at 8192 tokens
        {"name": "bwd_train", "op": "linear_bwd", "M": 8192, "N": 4096, "K": 4096},
        # decoding through 64 experts: a few rows each, most weights read once
        {"name": "moe_decode", "op": "grouped_fwd", "M": 96, "N": 2048, "K": 7168, "G": 64, "route": "zipf"},
        # a training batch through 8 unevenly loaded experts
        {"name": "moe_fwd", "op": "grouped_fwd", "M": 16384, "N": 2048, "K": 4096, "G": 8, "route": "dirichlet"},
        # its backward
        {"name": "moe_bwd", "op": "grouped_bwd", "M": 16384, "N": 2048, "K": 4096, "G": 8, "route": "dirichlet"},
        # the largest layer: 64 experts
        {"name": "moe_bwd_large", "op": "grouped_bwd", "M": 32768, "N": 2048, "K": 7168, "G": 64, "route": "zipf"},
        # adapters: many small tensors, launch-bound
        {"name": "adamw_adapters", "op": "adamw", "bits": 32, "tensors": 48, "rows": 2048, "cols": 16, "grad": "bf16",
         "copy": False},
        # the eight experts' weights and their biases, fp32 moments, a bf16 copy of the weights for the next step
        {"name": "adamw_experts", "op": "adamw", "bits": 32, "tensors": 8, "rows": 2048, "cols": 4096, "grad": "bf16",
         "copy": True},
        # the same with 8-bit moments
        {"name": "adamw8_experts", "op": "adamw", "bits": 8, "tensors": 8, "rows": 2048, "cols": 4096, "grad": "bf16",
         "copy": True},
    ]


def _log(rng, lo, hi, mul=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v) // mul * mul))


def draw(rng):
    op = rng.choice(["linear_fwd", "linear_bwd", "grouped_fwd", "grouped_bwd", "adamw"])
    if op == "adamw":
        tensors, rows = _log(rng, 1, 200), _log(rng, 16, 8192)
        cols = _log(rng, 1, max(2, min(8192, (1 << 26) // (tensors * rows))))
        return {"op": op, "bits": rng.choice([8, 32]), "tensors": tensors, "rows": rows, "cols": cols,
                "grad": rng.choice(["bf16", "f32"]), "copy": rng.random() < 0.5}
    while True:
        c = {"op": op, "M": _log(rng, 1, 32768), "N": _log(rng, 128, 8192, 16), "K": _log(rng, 128, 8192, 16)}
        if op.startswith("grouped"):
            c["G"] = _log(rng, 1, 128)
            c["route"] = rng.choice(["zipf", "dirichlet", "even"])
        big = c.get("G", 1) * c["N"] * c["K"]
        if c["M"] * c["N"] * c["K"] <= 1 << 37 and big <= 1 << 29:
            return c


def _ends(case):
    """Cumulative ends of the groups: expert loads by the case's routing, the same for every seed."""
    G, M = case.get("G", 1), case["M"]
    g = torch.Generator().manual_seed(1000 + G + M)
    if case.get("route") == "zipf":
        p = torch.arange(1, G + 1, dtype=torch.float64).pow(-1.1)[torch.randperm(G, generator=g)]
    elif case.get("route") == "dirichlet":
        p = -torch.rand(G, generator=g, dtype=torch.float64).clamp_min(1e-12).log()
    else:
        p = torch.ones(G, dtype=torch.float64)
    pick = torch.multinomial(p, M, replacement=True, generator=g)
    return torch.bincount(pick, minlength=G).cumsum(0).tolist()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if case["op"] == "adamw":
        return _prepare_adamw(case, randn)
    M, N, K, G = case["M"], case["N"], case["K"], case.get("G", 1)
    ends = _ends(case)
    s = {"op": case["op"], "ends": ends, "offsets": torch.tensor(ends, dtype=torch.int32, device="cuda")}
    w = torch.empty(G, N, K, dtype=torch.uint8, device="cuda")
    ws = torch.empty(G, -(-N // RUN), -(-K // RUN), device="cuda")
    for g in range(G):
        w[g], ws[g] = _quant_blocks(randn(N, K).mul_(0.02).bfloat16().float())
    s["w"], s["w_scales"] = w, ws
    # activations with a few outlier channels; gradients small and heavier-tailed along the tokens
    x = (randn(M, K) * (1 + 9 * (torch.rand(K, generator=gen, device="cuda") < 0.01))).bfloat16()
    if case["op"].endswith("fwd"):
        s["x"] = x
    else:
        v, sc = _quant_tokens(x.float(), s["offsets"])
        s["x_codes"], s["x_scales"] = v.to(F8).view(torch.uint8), sc
        s["grad"] = (randn(M, N) * 1e-3 * randn(M, 1).mul_(0.5).exp_()).bfloat16()
    return s


def _prepare_adamw(case, randn):
    """Matrices (decayed) then as many odd-length vectors (not decayed), every
    tensor at the start of a run of 128 of one flat buffer."""
    T, n, nv = case["tensors"], case["rows"] * case["cols"], case["rows"] + 1
    pad = lambda k: -(-k // RUN) * RUN  # noqa: E731
    starts = [i * pad(n) for i in range(T)] + [T * pad(n) + i * pad(nv) for i in range(T)]
    sizes = [n] * T + [nv] * T
    total, cut = T * (pad(n) + pad(nv)), T * pad(n)
    live = torch.zeros(total, device="cuda")
    live[:cut].view(T, -1)[:, :n] = 1
    live[cut:].view(T, -1)[:, :nv] = 1
    p = randn(total).mul_(0.02).mul_(live)
    scale = randn(total // RUN, 1).mul_(2).exp_().expand(-1, RUN).reshape(-1)          # gradients differ by orders of magnitude
    g = randn(total).mul_(1e-4).mul_(scale).mul_(live)
    m = randn(total).mul_(3e-5).mul_(scale).mul_(live)
    r = randn(total).abs_().add_(0.05).mul_(8e-5).mul_(scale).mul_(live)
    s = {"op": "adamw", "bits": case["bits"], "cut": cut, "starts": starts, "sizes": sizes, "p": p,
         "g": g.bfloat16() if case["grad"] == "bf16" else g,
         "copy": torch.zeros(total, dtype=torch.bfloat16, device="cuda") if case["copy"] else None}
    if case["bits"] == 32:
        s["m"], s["v"] = m, r.square_()
    else:
        mq, s["m_scales"] = _quant_runs(m.view(-1, RUN))
        rq, s["v_scales"] = _quant_runs(r.view(-1, RUN), keep=True)
        s["m"], s["v"] = (q.to(F8).view(torch.uint8).view(-1) for q in (mq, rq))
        s["m_scales"], s["v_scales"] = s["m_scales"].view(-1), s["v_scales"].view(-1)
    return s


# ---------------------------------------------------------------- plain forms

def _scales(amax):
    return torch.div(amax.clamp_min(FLOOR), amax.new_full((), E4M3_MAX))


def _codes(t):
    """The E4M3 values nearest to t, saturating."""
    return t.clamp_(-E4M3_MAX, E4M3_MAX).to(F8).float()


def _quant_runs(x, keep=False):
    """Code values and scales of runs along the last dimension (of at most 128). keep: a positive value never becomes 0."""
    s = _scales(x.abs().amax(-1, keepdim=True))
    t = torch.div(x, s)
    if keep:
        t = torch.where(x > 0, t.clamp_min(2.0 ** -9), t)
    return _codes(t), s


def _quant_cols(x):
    """x [M, K] -> code values [M, K], scales [M, ceil(K / 128)]: runs along K."""
    M, K = x.shape
    nb = -(-K // RUN)
    q, s = _quant_runs(torch.nn.functional.pad(x, (0, nb * RUN - K)).view(M, nb, RUN))
    return q.view(M, nb * RUN)[:, :K], s.view(M, nb)


def _run_of_row(offsets, M):
    """The run index of every row: group g's runs start at first_row // 128 + g."""
    row = torch.arange(M, dtype=torch.int32, device=offsets.device)
    g = torch.searchsorted(offsets, row, right=True)
    first = torch.cat([offsets.new_zeros(1), offsets])[g]
    return (first // RUN + g + (row - first) // RUN).long()


def _quant_tokens(x, offsets):
    """x [M, K] -> code values [M, K], scales [M // 128 + G, K]: runs along the rows of each group (0 for a run with no row)."""
    M, K = x.shape
    run = _run_of_row(offsets, M)
    amax = x.new_full((M // RUN + offsets.numel(), K), -1.0).index_reduce_(0, run, x.abs(), "amax")
    s = torch.where(amax < 0, 0.0, _scales(amax))
    return _codes(torch.div(x, s[run])), s


def _quant_blocks(w):
    """w [N, K] -> E4M3 bytes, scales per 128 x 128 block."""
    N, K = w.shape
    nr, nc = -(-N // RUN), -(-K // RUN)
    pad = torch.nn.functional.pad(w, (0, nc * RUN - K, 0, nr * RUN - N))
    s = _scales(pad.abs().view(nr, RUN, nc, RUN).amax((1, 3)))
    return _codes(torch.div(w, _spread(s, N, K))).to(F8).view(torch.uint8), s


def _spread(s, N, K):
    return s.repeat_interleave(RUN, -2)[..., :N, :].repeat_interleave(RUN, -1)[..., :K]


def _decode(codes):
    return codes.view(F8).float()


def _plain_products(st):
    w = _decode(st["w"]) * _spread(st["w_scales"], *st["w"].shape[-2:])
    spans = list(zip([0] + st["ends"], st["ends"]))
    if st["op"].endswith("fwd"):
        q, s = _quant_cols(st["x"].float())
        x = q * s.repeat_interleave(RUN, 1)[:, :q.shape[1]]
        return {"y": torch.cat([x[a:b] @ w[g].t() for g, (a, b) in enumerate(spans)]).bfloat16()}
    grad = st["grad"].float()
    q, s = _quant_cols(grad)
    g1 = q * s.repeat_interleave(RUN, 1)[:, :q.shape[1]]
    q, s = _quant_tokens(grad, st["offsets"])
    run = _run_of_row(st["offsets"], grad.shape[0])
    g2 = q * s[run]
    x = _decode(st["x_codes"]) * st["x_scales"][run]
    return {"dx": torch.cat([g1[a:b] @ w[g] for g, (a, b) in enumerate(spans)]).bfloat16(),
            "dw": torch.stack([g2[a:b].t() @ x[a:b] for a, b in spans]).bfloat16()}


def _plain_adamw(st):
    p, g, bits = st["p"], st["g"].float(), st["bits"]
    if bits == 32:
        m, v = st["m"], st["v"]
    else:
        m = (_decode(st["m"]).view(-1, RUN) * st["m_scales"].view(-1, 1)).view(-1)
        v = (_decode(st["v"]).view(-1, RUN) * st["v_scales"].view(-1, 1)).view(-1).square_()
    m.mul_(BETA1).add_(g * (1 - BETA1))
    v.mul_(BETA2).add_((g * g).mul_(1 - BETA2))
    r = v.sqrt()
    if bits == 8:
        for state, q in (("m", _quant_runs(m.view(-1, RUN))), ("v", _quant_runs(r.view(-1, RUN), keep=True))):
            st[state].copy_(q[0].to(F8).view(torch.uint8).view(-1))
            st[state + "_scales"].copy_(q[1].view(-1))
    step = m / r.mul_(1 / math.sqrt(1 - BETA2 ** STEP)).add_(EPS)
    p[:st["cut"]].mul_(1 - LR * DECAY)
    p.sub_(step.mul_(LR / (1 - BETA1 ** STEP)))
    if st["copy"] is not None:
        st["copy"].copy_(p)
    return _adamw_outputs(st)


def _adamw_outputs(st):
    out = {"p": st["p"], "copy": st["copy"]}
    if st["bits"] == 32:
        out["m"], out["v"] = st["m"], st["v"]
    else:
        out["m"], out["sqrt_v"] = st["m"].view(F8), st["v"].view(F8)
        out["m_scales"], out["v_scales"] = st["m_scales"], st["v_scales"]
    return out


# ---------------------------------------------------------------- the framework's calls

def _own_products(st):
    import fp8_gemm_backward_amd as lp
    dense = not st["op"].startswith("grouped")
    w = lp.QTensor("fp8_b128", st["w"], st["w_scales"])
    if st["op"] == "linear_fwd":
        return {"y": lp.lp_linear_fwd_dyn(st["x"], w)}
    if st["op"] == "grouped_fwd":
        return {"y": lp.lp_grouped_fwd_dyn(st["x"], w, st["offsets"])}
    x = lp.QTensor("fp8_r128", st["x_codes"], st["x_scales"], axis=-2)
    if dense:
        g1, g2 = lp.lp_r128_quant_dual(st["grad"])
        dx, _ = lp.lp_linear_bwd(g1, None, w, need_dw=False)
        _, dw = lp.lp_linear_bwd(g2, x, None, need_dx=False)
        return {"dx": dx, "dw": dw.unsqueeze(0)}
    g1, g2 = lp.lp_r128_quant_dual(st["grad"], offsets=st["offsets"])
    dx, _ = lp.lp_grouped_bwd(g1, None, w, st["offsets"], need_dw=False)
    _, dw = lp.lp_grouped_bwd(g2, x, None, st["offsets"], need_dx=False)
    return {"dx": dx, "dw": dw}


def _own_adamw(st):
    import fp8_gemm_backward_amd as lp
    if "plan" not in st:                      # the tensors a program hands its optimizer once
        at = [slice(a, a + n) for a, n in zip(st["starts"], st["sizes"])]
        runs = [slice(a // RUN, a // RUN - (-n // RUN)) for a, n in zip(st["starts"], st["sizes"])]
        st["plan"] = lp.AdamWPlan(
            [st["p"][i] for i in at], [st["g"][i] for i in at], [st["m"][i] for i in at], [st["v"][i] for i in at],
            exp_avg_scales=[st["m_scales"][i] for i in runs] if st["bits"] == 8 else None,
            exp_avg_sq_scales=[st["v_scales"][i] for i in runs] if st["bits"] == 8 else None,
            copies=[st["copy"][i] for i in at] if st["copy"] is not None else None,
            weight_decay=[DECAY if a < st["cut"] else 0.0 for a in st["starts"]])
    lp.lp_adamw(st["plan"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, step=STEP)
    return _adamw_outputs(st)


def run(state):
    if state["op"] == "adamw":
        return _own_adamw(state) if own else _plain_adamw(state)
    return _own_products(state) if own else _plain_products(state)


# ---------------------------------------------------------------- work and exact results

def work(case):
    if case["op"] == "adamw":
        n = case["tensors"] * (case["rows"] * case["cols"] + case["rows"] + 1)
        state = 16 if case["bits"] == 32 else 4 + 16 / RUN          # both moments read and written
        return {"bytes": n * (8 + state + (2 if case["grad"] == "bf16" else 4) + (2 if case["copy"] else 0)),
                "flops": 14 * n}
    M, N, K = case["M"], case["N"], case["K"]
    ends = _ends(case)
    used = sum(b > a for a, b in zip([0] + ends, ends))              # an expert without a row is not read
    w = used * (N * K + 4 * (-(-N // RUN)) * (-(-K // RUN)))
    if case["op"].endswith("fwd"):
        return {"bytes": 2 * M * K + w + 2 * M * N, "flops": 2 * M * N * K}
    x = M * K + 4 * (M // RUN + 1) * K
    return {"bytes": 2 * M * N + w + x + 2 * M * K + 2 * case.get("G", 1) * N * K, "flops": 4 * M * N * K}


def _nearest_e4m3(t):
    """E4M3 rounding of 64-bit values from its definition: 3 mantissa bits, exponents from -6, ties to even, at most 448."""
    _, e = torch.frexp(t)
    unit = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return (torch.round(t / unit) * unit).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_run(v):
    """Decoded values of one group of runs v [..., up to 128]: the stated fp32 roundings, everything else in 64 bits."""
    s = (v.abs().amax(-1, keepdim=True).clamp_min(FLOOR) / E4M3_MAX).float().double()
    return _nearest_e4m3((v / s).float().double()), s


def _exact_blocks(a, dim):
    """a [rows, cols] in 64 bits, quantized in runs of 128 along dim and decoded, run by run."""
    out = torch.empty_like(a)
    for b in range(0, a.shape[dim], RUN):
        part = a.narrow(dim, b, min(RUN, a.shape[dim] - b))
        q, s = _exact_run(part.movedim(dim, -1))
        out.narrow(dim, b, part.shape[dim]).copy_((q * s).movedim(-1, dim))
    return out


def _exact_weight(codes, scales):
    w = codes.view(F8).double()
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            w[i * RUN:(i + 1) * RUN, j * RUN:(j + 1) * RUN] *= scales[i, j].double()
    return w


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(st)
    spans = list(zip([0] + st["ends"], st["ends"]))
    if case["op"].endswith("fwd"):
        y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
        for g, (a, b) in enumerate(spans):
            if b > a:
                y[a:b] = _exact_blocks(st["x"][a:b].double(), 1) @ _exact_weight(st["w"][g], st["w_scales"][g]).t()
        return {"y": y}
    dx = torch.zeros(case["M"], case["K"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(len(spans), case["N"], case["K"], dtype=torch.float64, device="cuda")
    for g, (a, b) in enumerate(spans):
        if b > a:
            grad = st["grad"][a:b].double()
            dx[a:b] = _exact_blocks(grad, 1) @ _exact_weight(st["w"][g], st["w_scales"][g])
            x = st["x_codes"][a:b].view(F8).double()
            for i in range(0, b - a, RUN):
                x[i:i + RUN] *= st["x_scales"][a // RUN + g + i // RUN].double()
            dw[g] = _exact_blocks(grad, 0).t() @ x
    return {"dx": dx, "dw": dw}


def _exact_adamw(st):
    d = torch.float64
    p, g, cut = st["p"].to(d), st["g"].to(d), st["cut"]
    if st["bits"] == 32:
        m, v = st["m"].to(d), st["v"].to(d)
    else:
        m = (st["m"].view(F8).to(d).view(-1, RUN) * st["m_scales"].to(d)[:, None]).view(-1)
        v = (st["v"].view(F8).to(d).view(-1, RUN) * st["v_scales"].to(d)[:, None]).view(-1) ** 2
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    step = (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)).sqrt() + EPS)
    p[:cut] *= 1 - LR * DECAY
    p -= LR * step
    out = {"p": p, "copy": p if st["copy"] is not None else None}
    if st["bits"] == 32:
        out["m"], out["v"] = m, v
        return out
    mq, ms = _exact_run(m.view(-1, RUN))
    r = v.sqrt().view(-1, RUN)
    rq, rs = _exact_run(r)
    rq = torch.where((r > 0) & (rq == 0), 2.0 ** -9, rq)
    out["m"], out["sqrt_v"] = mq.view(-1), rq.view(-1)
    out["m_scales"], out["v_scales"] = ms.view(-1), rs.view(-1)
    return out
